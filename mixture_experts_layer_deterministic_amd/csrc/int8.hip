// 8-bit integers: symmetric codes with one fp32 scale a row (activations: a token; weights: an
// output channel), the quantiser and the expert-grouped products.
//
// A row's scale is amax / 127 (1 for a row of zeros; an amax below 2^-110 counts as 2^-110, so that
// no quotient leaves fp32's normal numbers) and its codes are rne(127 v / amax), -127 .. 127. A row
// that holds a value that is not finite gets codes 0 and the scale NaN: a product is NaN in that
// row's (or channel's) results and nowhere else.
// The products add codes exactly, in 32-bit integers (K below 2^17: 128 * 128 * K fits), so their
// results do not depend on any order of summation, nor on the kernel chosen:
//   out[p, n] = bf16(sa[p] * sum_k a[p, k] b[e, n, k] * sb[e, n]).
#include <algorithm>
#include <cmath>

#include "common.h"
#include "kernels.h"
#include "ops.h"
#include "products.h"

namespace moe {
namespace {

// 127 v / amax is a tie between two codes or at least 2^-16 of itself away from one: with v = a 2^i
// and amax = b 2^j (a, b < 256) the distance is a multiple of 2^(i-j) / 2b, and 127 a / b 2^(i-j) is
// at most 254 a < 2^16 times that. Products with 127 / amax moved by 2^-19 of itself down and up,
// each error below 2^-22, therefore round to the same code, or are a tie's two neighbours, of which
// the even one is taken. The sum with 1.5 2^23 rounds to a whole number, whose low byte is the code.
struct I8Scale {
  float scale, lo, hi;
  bool finite;
};
MOE_DEV I8Scale i8_scale(uint32_t amax_bits) {  // the largest magnitude's bf16 bits
  I8Scale s;
  s.finite = amax_bits < 0x7f80;
  float amax = __uint_as_float(amax_bits << 16);
  if (amax > 0.f) amax = fmaxf(amax, 0x1p-110f);
  const float inv = amax > 0.f && s.finite ? 127.f / amax : 0.f;
  s.scale = !s.finite ? __uint_as_float(0x7fc00000u) : amax > 0.f ? amax / 127.f : 1.f;
  s.lo = inv * (1.f - 0x1p-19f);
  s.hi = inv * (1.f + 0x1p-19f);
  return s;
}
MOE_DEV uint32_t i8_code(float v, const I8Scale& s) {
  const uint32_t lo = __float_as_uint(__builtin_fmaf(v, s.lo, 12582912.f));
  const uint32_t hi = __float_as_uint(__builtin_fmaf(v, s.hi, 12582912.f));
  return lo & 1 ? hi : lo;
}
MOE_DEV uint32_t i8_code4(float a, float b, float c, float d, const I8Scale& s) {
  const uint32_t ab = __builtin_amdgcn_perm(i8_code(b, s), i8_code(a, s), 0x0c0c0400u);
  const uint32_t cd = __builtin_amdgcn_perm(i8_code(d, s), i8_code(c, s), 0x0c0c0400u);
  return ab | cd << 16;
}
MOE_DEV uint2 i8_codes8(const uint4& x, const I8Scale& s) {
  if (!s.finite) return make_uint2(0, 0);
  return make_uint2(i8_code4(bf2f_lo(x.x), bf2f_hi(x.x), bf2f_lo(x.y), bf2f_hi(x.y), s),
                    i8_code4(bf2f_lo(x.z), bf2f_hi(x.z), bf2f_lo(x.w), bf2f_hi(x.w), s));
}
// The largest magnitude bits of eight bf16 values (they order as the magnitudes; NaN last).
MOE_DEV uint32_t amax_bits8(const uint4& x) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  u16x2 m = {0, 0};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[q] & 0x7fff7fffu));
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

// W waves take a row, U pieces of eight values a lane, all in registers: one read, past the caches.
// U = 0: rows too long for that are read twice. HBM bounds it, two thirds of it reads: 16384 x 7168 in
// 55 us, 6.4 TB/s, and 57344 x 2048 in 55.
template <int W, int U>
__global__ void __launch_bounds__(256) i8_quant_rows_kernel(const uint16_t* __restrict__ src,
                                                            long long rows, int cols,
                                                            uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
  constexpr int kPer = 4 / W;  // rows a workgroup
  __shared__ uint32_t red[4];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const long long r = (long long)blockIdx.x * kPer + wave / W;
  if (W == 1 && r >= rows) return;  // a whole wave; with W == 4 the grid has the rows
  const uint16_t* p = src + (size_t)r * cols;
  uint8_t* q = codes + (size_t)r * cols;
  const int c0 = (wave % W * kWave + lane) * 8;
  constexpr int kStep = W * kWave * 8;
  uint4 x[U ? U : 1];
  uint32_t amax = 0;
  if constexpr (U > 0) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      x[i] = c0 + i * kStep < cols ? nt_load16(p + c0 + i * kStep) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < U; ++i) amax = max(amax, amax_bits8(x[i]));
  } else {
    // unsigned: a row may end less than a step below 2^31
    for (uint32_t c = c0; c < (uint32_t)cols; c += kStep)
      amax = max(amax, amax_bits8(*reinterpret_cast<const uint4*>(p + c)));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, o));
  if constexpr (W > 1) {
    if (lane == 0) red[wave] = amax;
    __syncthreads();
    amax = max(max(red[0], red[1]), max(red[2], red[3]));
  }
  const I8Scale s = i8_scale(amax);
  if (wave % W == 0 && lane == 0) scales[r] = s.scale;
  if constexpr (U > 0) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (c0 + i * kStep < cols)
        *reinterpret_cast<uint2*>(q + c0 + i * kStep) = i8_codes8(x[i], s);
  } else {
    for (uint32_t c = c0; c < (uint32_t)cols; c += kStep)
      *reinterpret_cast<uint2*>(q + c) = i8_codes8(*reinterpret_cast<const uint4*>(p + c), s);
  }
}

// ------------------------------------------------------------------------------------------
// The products

// Where an epilogue finds its scales: in memory, at any multiple of 4 bytes, or in LDS. row(m): of
// the tile's row m; col(c): of four consecutive columns, c counting from the tile's first (a gated
// tile's up columns from up on).
MOE_DEV f32x4 col_scales(const float* p) { return f32x4{p[0], p[1], p[2], p[3]}; }
struct I8ScalesMem {
  const float *sa, *sb;
  int rows, up;
  MOE_DEV I8ScalesMem(const I8GemmArgs& a, int e, int row0, int rows_, int n0)
      : sa(a.sa + row0), sb(a.sb + (size_t)e * a.N + n0), rows(rows_), up(a.N / 2) {}
  MOE_DEV float row(int m) const { return sa[min(m, rows - 1)]; }
  MOE_DEV f32x4 col(int c) const { return col_scales(sb + c); }
};
// 256 rows' and 256 columns' scales of a 256 x 256 tile, in a KB each behind the tiles' units; waves
// 0..3 fetch the rows', waves 4..7 the columns' (gated: 128 of the gate, then the up projection's).
struct I8ScalesLds {
  static constexpr int up = 128;
  const float* st;
  template <bool GATED>
  static MOE_DEV void fetch(const I8GemmArgs& a, int e, int row0, int rows, int n0, uint8_t* to) {
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), i = wave % 4 * 64 + lane;
    const bool of_rows = wave < 4;
    const float* p = of_rows ? a.sa + row0 : a.sb + (size_t)e * a.N + n0;
    const int n = of_rows ? i : GATED && i >= 128 ? a.N / 2 + i - 128 : i;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        raw_rsrc(p, 4u * (of_rows ? rows : a.N - n0)),
        (__attribute__((address_space(3))) void*)(to + wave * 256), 4, 4u * n, 0, 0, 0);
  }
  MOE_DEV float row(int m) const { return st[m]; }
  MOE_DEV f32x4 col(int c) const { return *reinterpret_cast<const f32x4*>(st + 256 + c); }
};
// Rows row0 .. of the tile and columns n0 .. of its weights; a gated tile's n0 counts gate columns.
template <bool GATED, class T, class S>
MOE_DEV void i8_epilogue(const I8GemmArgs& a, const T& w, const S& sc, int row0, int rows, int n0,
                         int cols) {
  const int out_n = GATED ? a.N / 2 : a.N;
  if constexpr (!GATED) {
    const int c0 = w.wn * T::NB * 16;
    if (c0 >= cols) return;  // a whole wave
    f32x4 sb[T::NB];
#pragma unroll
    for (int nb = 0; nb < T::NB; ++nb) sb[nb] = sc.col(c0 + nb * 16 + 4 * (w.lane / 16));
#pragma unroll
    for (int mb = 0; mb < T::MB; ++mb) {
      const int m = w.row_of(mb);
      const bool on = m < rows;
      const float s = sc.row(m);
      f32x4 v[T::NB];
#pragma unroll
      for (int nb = 0; nb < T::NB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[nb][r] = (float)w.acc[mb][nb][r] * s * sb[nb][r];
      store_blocks<T::NB>(a.out + (size_t)(row0 + m) * out_n + n0 + c0, v, w.lane, on, false);
    }
  } else {
    constexpr int NG = T::NB / 2;
    const int c0 = w.wn * NG * 16;
    f32x4 sg[NG], su[NG];
#pragma unroll
    for (int nb = 0; nb < NG; ++nb) {
      sg[nb] = sc.col(c0 + nb * 16 + 4 * (w.lane / 16));
      su[nb] = sc.col(sc.up + c0 + nb * 16 + 4 * (w.lane / 16));
    }
    with_act(a.act, [&](auto tag) {
#pragma unroll
      for (int mb = 0; mb < T::MB; ++mb) {
        const int m = w.row_of(mb);
        const bool on = m < rows;
        const float s = sc.row(m);
        f32x4 v[NG];
#pragma unroll
        for (int nb = 0; nb < NG; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float g = (float)w.acc[mb][nb][r] * s * sg[nb][r];
            const float u = (float)w.acc[mb][nb + NG][r] * s * su[nb][r];
            v[nb][r] = act_of<decltype(tag)::value>(g) * u;
          }
        store_blocks<NG>(a.out + (size_t)(row0 + m) * out_n + n0 + c0, v, w.lane, on, false);
      }
    });
  }
}

struct I8Place {
  int e, row0, rows, n0;  // rows <= 0: none
};
template <bool GATED, class T>
MOE_DEV int i8_cols(const I8GemmArgs& a, const I8Place& t) {  // a plain tile's: its width, or 128
  return GATED ? T::BN : min(T::BN, a.N - t.n0);
}
template <bool GATED, class T>
MOE_DEV void i8_layout(const I8GemmArgs& a, T& w) {
  w.begin();
  w.a_rows(a.K);
  const int I = a.N / 2;
  w.b_rows(a.K, [&](int i) { return !GATED || i < T::BN / 2 ? i : I + i - T::BN / 2; });
}
template <class T>
MOE_DEV void i8_next(const I8GemmArgs& a, T& w, const I8Place& t) {
  w.next(a.a + (size_t)t.row0 * a.K, (uint32_t)t.rows * a.K,
         a.b + ((size_t)t.e * a.N + t.n0) * a.K, (uint32_t)(a.N - t.n0) * a.K);
}
template <int BM, int BN, bool GATED>
MOE_DEV void i8_tile(const I8GemmArgs& a, const I8Place& t) {
  using T = Tile8<Int8, BM, BN, false, false, GATED>;
  T w;
  i8_layout<GATED>(a, w);
  i8_next(a, w, t);
  w.run(a.K / 128);
  const I8ScalesMem sc(a, t.e, t.row0, t.rows, t.n0);
  i8_epilogue<GATED>(a, w, sc, t.row0, t.rows, t.n0, i8_cols<GATED, T>(a, t));
}

// Many rows an expert: 256 x 256 tiles, whole rounds of one a CU and then what is left, cut in two
// (256 x 128) or four (128 x 128) where the parts still fit one round. FLOW, where K has an even number
// of steps: a workgroup stays for all its tiles, and the next tile's first loads go out in the last
// steps of the one before, so that they arrive under its epilogue; otherwise each tile is a workgroup's.
//
// 16384 rows over 5 of 8 experts, gated 4096 x 7168: 360 us, 2.7e15 operations a second; 7168 x 2048:
// 230 us, 2.1e15 (a library product of one expert's 16384 rows, int32 results and no scales, takes 426
// and 247 us; this kernel 335 and 196 there). What bounds a step stands in
// products.h. With each tile a workgroup of its own the second took 238.
template <bool GATED, bool FLOW>
__global__ void __launch_bounds__(512, 2) i8_big_kernel(const I8GemmArgs a) {
  constexpr int kCols = GATED ? kBigT / 2 : kBigT;  // output columns
  const int nN = (a.N + kBigT - 1) / kBigT;
  const int nm = big_count(a), tiles = nm * nN;
  const int left = tiles % kCus, whole = tiles - left;
  const int cut = left * 4 <= kCus ? 4 : left * 2 <= kCus ? 2 : 1;
  const auto place = [&](int lt) {
    const int2 mn = big_order(lt, nm, nN);
    const RowTile t = big_rows(a, mn.x);
    return I8Place{t.e, t.row0, t.rows, mn.y * kCols};
  };
  // An XCD's tiles are contiguous; the round after the whole ones takes those that are left.
  int b = blockIdx.x;
  if constexpr (!FLOW) {
    if (b < whole) {
      i8_tile<256, 256, GATED>(a, place(xcd_contiguous(b, whole)));
      return;
    }
    b -= whole;
  }
  const int n8 = (left * cut + kXcds - 1) / kXcds * kXcds, j = xcd_contiguous(b, n8);
  const bool part = b < n8 && j < left * cut;
  if constexpr (FLOW) {
    const int rounds = whole / kCus + (cut == 1 && part ? 1 : 0);
    const auto at_round = [&](int r) {
      return place(r * kCus < whole ? xcd_contiguous(r * kCus + b, whole) : whole + j);
    };
    if (rounds > 0) {
      using T = Tile8<Int8, 256, 256, false, false, GATED>;
      T w;
      i8_layout<GATED>(a, w);
      I8Place t = at_round(0);
      i8_next(a, w, t);
      uint8_t* const st = prod_unit<8>();  // the tile's scales, then the next one's
      I8ScalesLds::fetch<GATED>(a, t.e, t.row0, t.rows, t.n0, st);
      loads_in_order();
      w.start(a.K / 128);
      for (int r = 0;; ++r) {
        I8Place n = t;
        if (r + 1 < rounds) n = at_round(r + 1);
        i8_next(a, w, n);
        w.template sum<true>();
        const I8ScalesLds sc{reinterpret_cast<const float*>(st + r % 2 * 2048)};
        i8_epilogue<GATED>(a, w, sc, t.row0, t.rows, t.n0, i8_cols<GATED, T>(a, t));
        I8ScalesLds::fetch<GATED>(a, n.e, n.row0, n.rows, n.n0, st + (r + 1) % 2 * 2048);
        if (r + 1 == rounds) break;
        t = n;
      }
      // the loads of a tile that does not come land before their places are given to another
      __builtin_amdgcn_s_waitcnt(kVm0Lgkm0);
      w.phase_end();
    }
  }
  if (!part || (FLOW && cut == 1)) return;
  I8Place t = place(whole + j / cut);
  if (!FLOW && cut == 1) {
    i8_tile<256, 256, GATED>(a, t);
    return;
  }
  t.n0 += j % cut % 2 * (kCols / 2);
  if (t.n0 >= (GATED ? a.N / 2 : a.N)) return;
  if (cut == 2) {
    i8_tile<256, 128, GATED>(a, t);
  } else {
    const int r = j % cut / 2 * 128;
    if (r >= t.rows) return;
    t.row0 += r;
    t.rows = min(t.rows - r, 128);
    i8_tile<128, 128, GATED>(a, t);
  }
}

// Few rows an expert: HBM bounds it. 256 experts of 64 rows, gated 4096 x 7168, in 1.33 ms, 5.8 TB/s; 24
// rows over 11 of 16 experts, 7168 x 2048, in 32 to 33 us, 5.0 TB/s.
template <int NMB, int SB, bool GATED>
MOE_DEV void i8_stream(const I8GemmArgs& a, const RowTile& t, int n0, const StreamStages<SB>& L) {
  StreamProduct<Int8, NMB, SB, GATED> w;
  w.begin();
  w.a_rows(a.a + (size_t)t.row0 * a.K, a.K, t.rows);
  const int I = a.N / 2;
  w.b_rows(a.b + (size_t)t.e * a.N * a.K, a.K, [&](int i) {
    return !GATED ? n0 + i : i < 64 ? n0 + i : I + n0 + i - 64;
  });
  w.run(L, a.K / 128);
  const I8ScalesMem sc(a, t.e, t.row0, t.rows, n0);
  i8_epilogue<GATED>(a, w, sc, t.row0, t.rows, n0, 128);
}
template <int BM, bool GATED>
__global__ void __launch_bounds__(256, BM == 128 ? 2 : 4) i8_stream_kernel(const I8GemmArgs a) {
  constexpr int SB = BM == 128 ? 3 : 2;
  __shared__ __align__(1024) uint8_t a0[BM * 128];
  __shared__ __align__(1024) uint8_t a1[BM * 128];
  __shared__ __align__(1024) uint8_t b0[128 * 128];
  __shared__ __align__(1024) uint8_t b1[128 * 128];
  __shared__ __align__(1024) uint8_t b2[SB == 3 ? 128 * 128 : 16];
  const StreamStages<SB> L{a0, a1, b0, b1, b2};
  const int nN = a.N / 128, lt = blockIdx.x;
  const RowTile t = find_rows<BM>(a.offsets, a.M, a.E, lt / nN);
  if (t.rows <= 0) return;  // whole workgroup
  const int n0 = lt % nN * (GATED ? 64 : 128);
  if (BM == 32 || t.rows <= 32) i8_stream<2, SB, GATED>(a, t, n0, L);
  else if (t.rows <= 64) i8_stream<4, SB, GATED>(a, t, n0, L);
  else if (t.rows <= 96) i8_stream<6, SB, GATED>(a, t, n0, L);
  else i8_stream<8, SB, GATED>(a, t, n0, L);
}

// A handful of experts with a handful of rows: a workgroup for 16 NNB rows of an expert's weights
// (gated: 8 NNB columns) and 16 NMB rows. One expert of 16 rows, gated 4096 x 7168: 11 us, 2.7 TB/s of
// weights.
template <int NMB, int NNB, int U, bool GATED>
__global__ void __launch_bounds__(512, NMB * NNB == 1 ? 4 : 2) i8_skinny_kernel(
    const I8GemmArgs a) {
  __shared__ i32x4 red[8 * NMB * NNB * kWave];
  const int nN = a.N / (16 * NNB), I = a.N / 2;
  const RowTile t = find_rows<16 * NMB>(a.offsets, a.M, a.E, blockIdx.x / nN);
  if (t.rows <= 0) return;  // whole workgroup
  const int n0 = blockIdx.x % nN * (GATED ? 8 : 16) * NNB;
  SkinnyProduct<Int8, NMB, NNB, U> w;
  w.begin();
  w.a_rows(a.a + (size_t)t.row0 * a.K, a.K, t.rows);
  w.b_rows(a.b + (size_t)t.e * a.N * a.K, a.K, [&](int i) {
    return !GATED ? n0 + i : n0 + i / 16 * 8 + (i % 16 < 8 ? i % 16 : I + i % 16 - 8);
  });
  w.run(a.K / 128, red);
  if (w.wave >= NMB * NNB) return;
  const int m = w.wave / NNB * 16 + w.lane % 16;
  const float s = a.sa[t.row0 + min(m, t.rows - 1)];
  const float* sb = a.sb + (size_t)t.e * a.N;
  const size_t row = t.row0 + m;
  if constexpr (!GATED) {
    const int c = n0 + w.wave % NNB * 16;
    const f32x4 sc = col_scales(sb + c + 4 * (w.lane / 16));
    f32x4 v[1];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[0][r] = (float)w.acc[0][0][r] * s * sc[r];
    store_blocks<1>(a.out + row * a.N + c, v, w.lane, m < t.rows, false);
  } else {
    // lanes 0..31 hold four gate columns of a row, lanes 32..63 the matching ups
    const int c = n0 + w.wave % NNB * 8 + 4 * (w.lane / 16 % 2);
    const f32x4 sc = col_scales(sb + (w.lane < 32 ? 0 : I) + c);
    f32x4 g, u;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      g[r] = (float)w.acc[0][0][r] * s * sc[r];
      u[r] = __shfl_xor(g[r], 32);
    }
    if (m >= t.rows || w.lane >= 32) return;
    with_act(a.act, [&](auto tag) {
      constexpr int A = decltype(tag)::value;
      *reinterpret_cast<uint2*>(a.out + row * I + c) =
          make_uint2(to_bf2(act_of<A>(g[0]) * u[0], act_of<A>(g[1]) * u[1]),
                     to_bf2(act_of<A>(g[2]) * u[2], act_of<A>(g[3]) * u[3]));
    });
  }
}

}  // namespace

hipError_t launch_i8_quant_rows(const uint16_t* src, long long rows, int cols, uint8_t* codes,
                                float* scales, hipStream_t s) {
  TraceScope trace("i8_quant_rows", s);
  const auto go = [&](auto kernel, int per) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, src, rows,
                       cols, codes, scales);
  };
  if (cols <= 512) go(i8_quant_rows_kernel<1, 1>, 4);
  else if (cols <= 1024) go(i8_quant_rows_kernel<1, 2>, 4);
  else if (cols <= 2048) go(i8_quant_rows_kernel<1, 4>, 4);
  else if (cols <= 4096) go(i8_quant_rows_kernel<1, 8>, 4);
  else if (cols <= 8192) go(i8_quant_rows_kernel<4, 4>, 1);
  else if (cols <= 16384) go(i8_quant_rows_kernel<4, 8>, 1);
  else go(i8_quant_rows_kernel<4, 0>, 1);
  return hipGetLastError();
}

template <int NMB, int NNB>
static void launch_skinny(const I8GemmArgs& a, bool gated, hipStream_t s) {
  const dim3 grid((unsigned)(a.M / (16 * NMB) + a.E) * (a.N / (16 * NNB)));
  if (gated)
    hipLaunchKernelGGL((i8_skinny_kernel<NMB, NNB, 4, true>), grid, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((i8_skinny_kernel<NMB, NNB, 4, false>), grid, dim3(512), 0, s, a);
}

// Which kernel, by the rows an expert has on average and the 128-row tiles of the weights there are
// (M, E and N are all the host knows of the load; every kernel is right for every load, and every
// kernel's results are the same). Measured in us a call, rows spread evenly, experts x rows, gated
// with N x K = 4096 x 7168 where not said:
//  * up to 64 tiles and few rows: every CU at the weights. 1 x 1 9 (128-row streaming 26), 1 x 16 11
//    (26), 1 x 64 18.5 (31), 2 x 16 19 (27). 2 x 64 34 (32), and 128 tiles, 4 x 16, 42 (29).
//  * 513 to 665 tiles with rows in them, up to 16 rows: 32-row streaming, whose second round is then
//    not nearly empty as that of two 128-row tiles a CU: 17 x 8 85 (94), 20 x 16 93 (112); 22 x 8 121
//    (113), 28 x 8 135 (125). The host counts the experts that have rows as if M rows were dealt at
//    random.
//  * up to 112 rows: 128-row streaming. 64 x 96 362 (256 x 256 tiles 401), 16 x 96 93 (103), 32 x 128
//    198 (210); from 129 rows on an expert's weights are read twice, 32 x 144 342 (214), and of experts
//    with 128 on average half have more. But 193 to 256 tiles (192 from 64 rows on) in halves of
//    256 x 256 tiles fill the card just once: 7 x 64 50 (61), 8 x 48 52 (58), 6 x 96 50 (69), 7168 x
//    4096 not gated 4 x 64 34 (38); 6 x 64 48 (37), 9 x 64 79 (64).
hipError_t launch_i8_gemm(const I8GemmArgs& a, bool gated, hipStream_t s) {
  auto grid = [&](int bm, int bn) {
    const unsigned n = (unsigned)(a.M / bm + a.E) * (unsigned)((a.N + bn - 1) / bn);
    return dim3((n + kXcds - 1) / kXcds * kXcds);
  };
  TraceScope trace(gated ? "i8_gemm_gated" : "i8_gemm", s);
  const long long M = a.M, E = a.E, tiles = E * (a.N / 128);
  if (tiles <= kCus / 4 && (M <= 32 * E || M <= 64)) {
    if (M <= 16 * E) launch_skinny<1, 1>(a, gated, s);
    else if (M <= 32 * E) launch_skinny<2, 1>(a, gated, s);
    else launch_skinny<2, 2>(a, gated, s);
    return hipGetLastError();
  }
  const double busy = (double)tiles * -std::expm1(-(double)M / (double)E);
  constexpr int kMost = 3 * kCus / 4;
  const bool once = tiles >= kMost && tiles <= kCus && M > (tiles > kMost ? 32 : 64) * E;
  if (busy > 2 * kCus && busy <= 2.6 * kCus && M <= 16 * E) {
    const auto kernel = gated ? i8_stream_kernel<32, true> : i8_stream_kernel<32, false>;
    hipLaunchKernelGGL(kernel, grid(32, 128), dim3(256), 0, s, a);
  } else if (M <= 112 * E && !once) {
    const auto kernel = gated ? i8_stream_kernel<128, true> : i8_stream_kernel<128, false>;
    hipLaunchKernelGGL(kernel, grid(128, 128), dim3(256), 0, s, a);
  } else {
    const bool flow = a.K / 128 % 2 == 0;  // two stages
    const auto kernel = gated ? (flow ? i8_big_kernel<true, true> : i8_big_kernel<true, false>)
                              : (flow ? i8_big_kernel<false, true> : i8_big_kernel<false, false>);
    // a workgroup a CU, or room for every tile and for a last round's parts
    const dim3 g = flow ? dim3(kCus) : dim3(grid(kBigT, kBigT).x + kCus);
    hipLaunchKernelGGL(kernel, g, dim3(512), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
