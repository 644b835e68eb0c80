// The gate: scores from the router logits, the choice of k experts per token, its weights, and
// the gradient of the logits.
//
// With s = softmax(l) or sigmoid(l) over a row of E logits and a balance bias b, the choice
// score is c = s + b. The experts form G equal runs (groups); a group scores the largest c it
// holds, or the sum of its two largest. The best `topk_groups` groups stay, then the k largest c
// in them are selected, ties to the lower index both times. The bias moves the choice only: the
// weights are w_j = scale * s_j, or scale * s_j / sum_i s_i over the selected.
// A logit of -inf (or NaN) closes its expert: it scores 0 and comes behind every open one.
//
// The choice is discontinuous, so it is made on 64-bit values: in 32 bits two rounded scores
// meet or swap where the definition keeps them apart. Where c orders as the logits do (no bias
// and no sums of scores) the logits themselves are compared, which is exact.
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "ops.h"

namespace moe {
namespace {

constexpr int kGateWaves = 4;
constexpr double kClosed = -1.7e308;  // below every open choice score, above what is taken

// x with lanes moved by a DPP control word; lanes without a source keep their own.
template <int CTRL, int ROWS>
MOE_DEV uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
MOE_DEV uint64_t dpp(uint64_t x) {
  return (uint64_t)dpp<CTRL, ROWS>((uint32_t)x) |
         ((uint64_t)dpp<CTRL, ROWS>((uint32_t)(x >> 32)) << 32);
}
template <int CTRL, int ROWS>
MOE_DEV float dpp(float x) {
  return __builtin_bit_cast(float, dpp<CTRL, ROWS>(__builtin_bit_cast(uint32_t, x)));
}
template <int CTRL, int ROWS>
MOE_DEV double dpp(double x) {
  return __builtin_bit_cast(double, dpp<CTRL, ROWS>(__builtin_bit_cast(uint64_t, x)));
}
MOE_DEV uint32_t read_lane(uint32_t x, int l) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, l);
}
MOE_DEV float read_lane(float x, int l) {
  return __builtin_bit_cast(float, read_lane(__builtin_bit_cast(uint32_t, x), l));
}
MOE_DEV double read_lane(double x, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, (uint64_t)read_lane((uint32_t)u, l) |
                                        ((uint64_t)read_lane((uint32_t)(u >> 32), l) << 32));
}
MOE_DEV uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
MOE_DEV float larger(float a, float b) { return fmaxf(a, b); }
MOE_DEV double larger(double a, double b) { return __builtin_fmax(a, b); }
// x moved likewise; lanes without a source get 0.
template <int CTRL, int ROWS>
MOE_DEV uint32_t dpp0(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, ROWS == 0xf);
}
template <int CTRL, int ROWS>
MOE_DEV float dpp0(float x) {
  return __builtin_bit_cast(float, dpp0<CTRL, ROWS>(__builtin_bit_cast(uint32_t, x)));
}
template <int CTRL, int ROWS>
MOE_DEV double dpp0(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, (uint64_t)dpp0<CTRL, ROWS>((uint32_t)u) |
                                        ((uint64_t)dpp0<CTRL, ROWS>((uint32_t)(u >> 32)) << 32));
}
// Over the wave, the same in every lane: within rows of 16 lanes by shifts, then lane 15's and
// lane 31's totals move on to the rows behind them.
template <class F>
MOE_DEV F wave_sum(F v) {
  v += dpp0<0x111, 0xf>(v);
  v += dpp0<0x112, 0xf>(v);
  v += dpp0<0x114, 0xf>(v);
  v += dpp0<0x118, 0xf>(v);
  v += dpp0<0x142, 0xa>(v);
  v += dpp0<0x143, 0xc>(v);
  return read_lane(v, 63);
}
// A maximum may meet a lane's own value again, so nothing has to be masked. Of unsigned numbers
// 0 is neutral: the shift then merges into the maximum, one instruction a step.
MOE_DEV uint32_t wave_max(uint32_t v) {
  v = max(v, dpp0<0x111, 0xf>(v));
  v = max(v, dpp0<0x112, 0xf>(v));
  v = max(v, dpp0<0x114, 0xf>(v));
  v = max(v, dpp0<0x118, 0xf>(v));
  v = max(v, dpp0<0x142, 0xa>(v));
  v = max(v, dpp0<0x143, 0xc>(v));
  return read_lane(v, 63);
}
template <class F>
MOE_DEV F wave_max(F v) {
  v = larger(v, dpp<0x111, 0xf>(v));
  v = larger(v, dpp<0x112, 0xf>(v));
  v = larger(v, dpp<0x114, 0xf>(v));
  v = larger(v, dpp<0x118, 0xf>(v));
  v = larger(v, dpp<0x142, 0xa>(v));
  v = larger(v, dpp<0x143, 0xc>(v));
  return read_lane(v, 63);
}
// exp(x) for the scores, x <= 709: e^x = 2^n e^r with n = rint(x / ln 2) and |r| <= ln(2) / 2,
// e^r by its Taylor polynomial. Degree 12 (the next term is below 1.8e-16) gives about 1e-15 in
// all, with 20 instructions; the library's exp also covers what does not occur here. Degree 10
// (2.2e-13, and |x| 2^-53 from one rounded ln 2) is for a sum that only divides what is then
// rounded to fp32.
template <int DEGREE = 12>
MOE_DEV double exp64(double x) {
  x = __builtin_fmax(x, -746.0);  // 2^-1076.2, which rounds to 0
  // adding 1.5 2^52 rounds to a whole number, which the sum's low word then holds
  const double t = __builtin_fma(x, 1.4426950408889634, 6755399441055744.0);
  const double n = t - 6755399441055744.0;
  double r;
  if constexpr (DEGREE == 12) {  // ln 2 cut to 33 bits, n times which is exact, and the rest
    r = __builtin_fma(n, -6.93147180369123816490e-01, x);
    r = __builtin_fma(n, -1.90821492927058770002e-10, r);
  } else {
    r = __builtin_fma(n, -6.93147180559945309417e-01, x);
  }
  double p = DEGREE == 12 ? 1.0 / 479001600.0 : 1.0 / 3628800.0;
  if constexpr (DEGREE == 12) {
    p = __builtin_fma(p, r, 1.0 / 39916800.0);
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
  }
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)__builtin_bit_cast(uint64_t, t));
}
// 1 / y for normal y, to about one step: two Newton steps on the hardware's estimate.
MOE_DEV double rcp64(double y) {
  double r = __builtin_amdgcn_rcp(y);
  r = __builtin_fma(__builtin_fma(-y, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-y, r, 1.0), r, r);
}

// Softmax numerator of logit l under the row's largest m: 1 at the largest (so +inf entries
// share the row), 0 for a closed expert and in a row that holds nothing else.
MOE_DEV double soft_num64(float l, float m) {
  const double x = exp64((double)l - (double)m);  // no branch: the constants stay in registers
  return l == -INFINITY ? 0.0 : l == m ? 1.0 : x;
}
MOE_DEV float soft_num(float l, float m) {
  return l == -INFINITY ? 0.f : l == m ? 1.f : expf(l - m);
}
MOE_DEV double sigmoid64(float l) {
  // below -709 the sum leaves 64 bits' range and the score is 0
  const double x = rcp64(1.0 + exp64(-(double)fmaxf(l, -709.f)));
  return l < -709.f ? 0.0 : x;
}

// a + b with b as it is stored otherwise: not fused with the product that made it.
MOE_DEV float add_rounded(float a, float b) {
#pragma clang fp contract(off)
  return a + b;
}

// fp32 in an order that unsigned integers compare, and back; 0 lies below every value's.
MOE_DEV uint32_t order32(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);  // -0 as +0
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
MOE_DEV float unorder32(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The same for 64-bit scores.
MOE_DEV uint64_t order64(double c) {
  const uint64_t u = __builtin_bit_cast(uint64_t, c);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
MOE_DEV uint32_t upper(uint32_t x) { return x; }
MOE_DEV uint32_t upper(uint64_t x) { return (uint32_t)(x >> 32); }
MOE_DEV int count(uint64_t lanes) { return __popcll(lanes); }
// What the wave's lanes wrote to LDS is read behind this by the same wave.
MOE_DEV void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// hit[v]: the lanes whose key[v] is a candidate. All k largest keys of the wave (ties to the lower
// lane, then slot) are among the candidates, which are 64 at most; their number is returned.
// Keys whose upper half lies below `least` are none. At least k keys are not such.
//
// The k-th largest of the lanes' own maxima bounds the k-th largest key from below, and few keys
// lie above it. From the largest maximum down by steps that grow, then by halves, over the upper
// 32 bits, a search finds a bound that k to k + 4 maxima reach: a compare and scalar instructions
// a step. Where that leaves more than 64 keys (equal ones, or all in few lanes), the k-th key and
// then its index are found exactly, bit by bit.
template <int V, class U>
MOE_DEV int pick_candidates(const U (&key)[V], uint32_t least, int k, int lane,
                            uint64_t (&hit)[V]) {
  uint32_t head = upper(key[0]);
#pragma unroll
  for (int v = 1; v < V; ++v) head = max(head, upper(key[v]));
  uint32_t hi = wave_max(head) + 1, lo, step = sizeof(U) == 4 ? 1u << 20 : 1u << 17;
  int more;     // maxima that reach lo, less k
  while (true) {  // an eighth of a binade, a half, two, eight, 32, ..
    lo = hi - least > step ? hi - step : least;
    more = count(__ballot(head >= lo)) - k;
    if (more >= 0 || lo == least) break;
    hi = lo;
    step = step < 1u << 29 ? step * 4 : step;
  }
  while (more > 4 && hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int n = count(__ballot(head >= mid)) - k;
    if (n < 0) {
      hi = mid;
    } else {
      lo = mid;
      more = n;
    }
  }
  int total = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    hit[v] = __ballot(upper(key[v]) >= lo);
    total += count(hit[v]);
  }
  if (total <= kWave) return total;
  U kth = 0;  // the largest value that k keys reach
  for (int b = 8 * sizeof(U) - 1; b >= 0; --b) {
    const U x = kth | U(1) << b;
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) n += count(__ballot(key[v] >= x));
    if (n >= k) kth = x;
  }
  int above = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) above += count(__ballot(key[v] > kth));
  int end = 0;  // the largest index in front of which too few are equal to it
  for (int b = 9; b >= 0; --b) {
    const int x = end | 1 << b;
    int n = above;
#pragma unroll
    for (int v = 0; v < V; ++v) n += count(__ballot(key[v] == kth && lane * V + v < x));
    if (n < k) end = x;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    hit[v] = __ballot(key[v] > kth || (key[v] == kth && lane * V + v <= end));
  return k;
}

// One wave per token: lane l holds the V experts from V l on. pick_candidates leaves at most 64,
// mostly little more than k; each then counts those in front of it, all against all, which is its
// place among the choices.
// LOGIT: the scores order as the logits do; 32-bit keys, and 64-bit scores only of the chosen.
// Groups that are whole, aligned runs of 2^i lanes are scored by lane exchanges, others in LDS.
//
// 18944 x 512, softmax, k = 10: 19.2 us (the profiler's median; 16.7 a call in a run of calls), 2.0
// TB/s of logits. Vector issue bounds it (460 instructions a token, a third of them the row's
// 64-bit exponentials; 85 - 90% of the time). 16, 2048 and 18944 tokens of 256 with 8 groups,
// sigmoid and bias: 4.9 and 6.1 us, a chain of latencies, and 23.4 (21.9 a call), vector issue
// again: a 64-bit exponential and reciprocal for every expert. k rounds of the wave's maximum over
// lanes of sorted keys, in place of the list, took 23.6 a call where this takes 16.7, and 5.3, 6.8
// and 29.4.
template <int V, bool LOGIT>
__global__ void __launch_bounds__(kGateWaves* kWave) gate_select_kernel(
    GateParams p, const float* __restrict__ logits, const float* __restrict__ bias, int T, int E,
    int k, int vec, int32_t* __restrict__ idx, float* __restrict__ w) {
  using C = std::conditional_t<LOGIT, uint32_t, double>;
  constexpr C kTaken = LOGIT ? C(0) : C(-INFINITY);
  extern __shared__ double gate_lds[];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int t = blockIdx.x * kGateWaves + wave;
  const bool live = t < T;
  const int e0 = lane * V;
  const float* row = logits + (size_t)(live ? t : 0) * E;
  float l[V];
  if (V >= 4 && vec) {  // rows of whole 16-byte pieces
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      const f32x4 x = e0 + v < E ? *reinterpret_cast<const f32x4*>(row + e0 + v)
                                 : f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 4 && v + i < V; ++i) l[v + i] = x[i];
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? row[e0 + v] : -INFINITY;
  }
  float m = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    l[v] = l[v] == l[v] ? l[v] : -INFINITY;
    m = fmaxf(m, l[v]);
  }
  double zi = 0;  // 1 / sum of the softmax numerators (0 for a row of closed experts)
  if (p.softmax) {
    m = wave_max(m);
    if (!LOGIT || !p.renorm) {  // renormalised weights need no sum over the row
      double z = 0;
      if (m == INFINITY) {  // for the whole wave: the +inf entries share the row
#pragma unroll
        for (int v = 0; v < V; ++v) z += l[v] == INFINITY ? 1.0 : 0.0;
      } else {  // a closed expert's is 0
#pragma unroll
        for (int v = 0; v < V; ++v) z += exp64<LOGIT ? 10 : 12>((double)l[v] - (double)m);
      }
      z = wave_sum(z);
      zi = m > -INFINITY ? rcp64(z) : 0.0;
    }
  }
  // Places past the row's end count as closed experts: of equals they come last, and k <= E.
  C c[V];
  double sv[LOGIT ? 1 : V];  // the scores, 0 of closed experts
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (LOGIT) {
      c[v] = order32(l[v]);
    } else {
      const double s = !p.softmax      ? sigmoid64(l[v])
                       : m == INFINITY ? (l[v] == INFINITY ? zi : 0.0)
                                       : exp64((double)l[v] - (double)m) * zi;
      const double x = s + (bias ? (double)bias[min(e0 + v, E - 1)] : 0.0);
      c[v] = l[v] > -INFINITY && x > kClosed ? x : kClosed;
      sv[v] = l[v] > -INFINITY ? s : 0.0;
    }
  }
  // groups
  const int G = p.groups, gs = E / G;
  if (G > 1 && p.topk_groups < G) {  // the same for the whole grid
    const int lpg = gs / V;
    if (gs % V == 0 && (lpg & (lpg - 1)) == 0) {
      C a = c[0], b = kTaken;  // the lane's two largest, then its group's
#pragma unroll
      for (int v = 1; v < V; ++v) {
        const C lo = c[v] > a ? a : c[v];
        a = larger(a, c[v]);
        b = larger(b, lo);
      }
      auto merge = [&](C a1, C b1) {
        const C lo = a1 > a ? a : a1;
        a = larger(a, a1);
        b = larger(larger(b, b1), lo);
      };
      // lane l with l ^ 1, l ^ 2, then mirrored in 8 and in 16 lanes, whose halves agree by then
      if (lpg > 1) merge(dpp<0xb1, 0xf>(a), dpp<0xb1, 0xf>(b));
      if (lpg > 2) merge(dpp<0x4e, 0xf>(a), dpp<0x4e, 0xf>(b));
      if (lpg > 4) merge(dpp<0x141, 0xf>(a), dpp<0x141, 0xf>(b));
      if (lpg > 8) merge(dpp<0x140, 0xf>(a), dpp<0x140, 0xf>(b));
      for (int o = 16; o < lpg; o <<= 1) merge(__shfl_xor(a, o), __shfl_xor(b, o));
      if constexpr (!LOGIT)
        if (p.top2 && b > kClosed) a += b;
      const int mine = lane / lpg;
      int rank = 0;  // groups that go before this lane's
      for (int g = 0; g < G; ++g) {
        const C o = read_lane(a, g * lpg);
        rank += o > a || (o == a && g < mine);
      }
      if (mine >= G || rank >= p.topk_groups) {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = kTaken;
      }
    } else {
      double* cs = gate_lds + (size_t)wave * (E + G);
      double* gsc = cs + E;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e0 + v < E) cs[e0 + v] = (double)c[v];
      __syncthreads();
      for (int g = lane; g < G; g += kWave) {
        double a = -INFINITY, b = -INFINITY;
        for (int i = 0; i < gs; ++i) {
          const double x = cs[g * gs + i];
          const double lo = x > a ? a : x;
          a = larger(a, x);
          b = larger(b, lo);
        }
        if constexpr (!LOGIT)
          if (p.top2 && b > kClosed) a += b;
        gsc[g] = a;
      }
      __syncthreads();
      uint32_t stay = 0;  // bit i: group lane + 64 i
      for (int i = 0; lane + kWave * i < G; ++i) {
        const int g = lane + kWave * i;
        const double a = gsc[g];
        int rank = 0;
        for (int h = 0; h < G; ++h) {
          const double o = gsc[h];
          rank += o > a || (o == a && h < g);
        }
        if (rank < p.topk_groups) stay |= 1u << i;
      }
      __syncthreads();
      for (int i = 0; lane + kWave * i < G; ++i) gsc[lane + kWave * i] = (stay >> i) & 1u;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e0 + v >= E || gsc[(e0 + v) / gs] == 0.0) c[v] = kTaken;
    }
  }
  // the candidates side by side in LDS, one a lane, in the order of their slots
  using U = std::conditional_t<LOGIT, uint32_t, uint64_t>;
  U key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (LOGIT) key[v] = c[v];
    else key[v] = order64(c[v]);
  }
  uint64_t hit[V];
  const int n = pick_candidates(key, LOGIT ? 1u : upper(order64(kClosed)), k, lane, hit);
  // LOGIT: the key and the index's complement in one number. Else the list is in index order, so
  // equal keys are in the order of their places.
  __shared__ __align__(16) uint64_t list[kGateWaves][kWave];
  __shared__ double list_s[LOGIT ? 1 : kGateWaves][kWave];
  __shared__ int list_e[LOGIT ? 1 : kGateWaves][kWave];
  list[wave][lane] = 0;
  wave_sync();
  int at = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
    at = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(hit[v] >> 32),
                                        __builtin_amdgcn_mbcnt_lo((uint32_t)hit[v], at));
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (__builtin_amdgcn_inverse_ballot_w64(hit[v])) {
      if constexpr (LOGIT) {
        list[wave][at] = (uint64_t)key[v] << 32 | (uint32_t)~(e0 + v);
      } else {
        list[wave][at] = key[v];
        list_s[wave][at] = sv[v];
        list_e[wave][at] = e0 + v;
      }
      ++at;
    }
  }
  wave_sync();
  // a candidate's place is the number of those in front of it
  const uint64_t mine = list[wave][lane];
  int place = 0;
  constexpr int kStep = LOGIT ? 4 : 8;  // fewer compares past n; fewer waits
#pragma unroll 1
  for (int j = 0; j < n; j += kStep) {
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      const uint64_t o = list[wave][j + i];
      if constexpr (LOGIT) place += o > mine;
      else place += o > mine || (o == mine && j + i < lane);
    }
  }
  const bool chosen = lane < n && place < k;
  int my_e = 0;
  double s = 0;  // the score, 0 where nothing was chosen
  if (chosen) {
    if constexpr (LOGIT) {
      my_e = (int)~(uint32_t)mine;
      const float my_l = unorder32(upper(mine));
      s = !p.softmax ? sigmoid64(my_l) : soft_num64(my_l, m);
      if (p.softmax && zi > 0) s *= zi;
    } else {
      my_e = list_e[wave][lane];
      s = list_s[wave][lane];
    }
  }
  if (p.renorm) {
    const double sum = wave_sum(s);
    s = sum > 0 ? s / sum : 0.0;
  } else if (p.softmax && !(zi > 0)) {
    s = 0;
  }
  if (live && chosen) {
    idx[(size_t)t * k + place] = my_e;
    w[(size_t)t * k + place] = (float)(s * (double)p.scale);
  }
}

// One wave per token. Lane j < k takes slot j:
//   g_j = scale dw_j
//   sigmoid:                 dl_j = g_j s_j (1 - s_j)
//   sigmoid, renormalised:   dl_j = (g_j - sum_i g_i q_i) q_j (1 - s_j),  q = s / S
//   softmax, renormalised:   dl_j = q_j (g_j - sum_i q_i g_i)
//   softmax:                 dl_e = p_e ([e selected] g_e - sum_i p_i g_i), for every e
// The slots' values are scattered over a row of zeros in LDS and the row leaves in 16-byte
// pieces. Slots that name one expert twice (found by each slot writing its number to its
// expert's place and reading it back) are added one after the other, in ascending j; a slot
// outside [0, E) counts nothing. DENSE, softmax without renorm, also reads the row of logits.
// 18944 x 512, every logit: 16.7 us, 4.7 TB/s, HBM's rate for as much read as written (a large copy
// does 4.65). 2048 x 256, sigmoid: 3.5 us, the launch and one chain of loads.
template <int V, bool DENSE>
__global__ void __launch_bounds__(kGateWaves* kWave) gate_backward_kernel(
    GateParams p, const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const float* __restrict__ dw, int T, int E, int k, int vec, float* __restrict__ dl,
    int accumulate) {
  __shared__ __align__(16) float rows[kGateWaves][V * kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int t = blockIdx.x * kGateWaves + wave;
  const bool live = t < T;
  const size_t tt = live ? t : 0;
  const float* row = logits + tt * E;
  float* out = dl + tt * E;
  const int e0 = lane * V;
  float l[V];
  if constexpr (DENSE) {
    if (V >= 4 && vec) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const f32x4 x = e0 + v < E ? *reinterpret_cast<const f32x4*>(row + e0 + v)
                                   : f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 4 && v + i < V; ++i) l[v + i] = x[i];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? row[e0 + v] : -INFINITY;
    }
  }
  int e = lane < k ? idx[tt * k + lane] : -1;
  if (e < 0 || e >= E) e = -1;
  float lj = e >= 0 ? row[e] : -INFINITY;
  lj = lj == lj ? lj : -INFINITY;
  const float g = e >= 0 ? p.scale * dw[tt * k + lane] : 0.f;
  float val, zi = 0.f, m = -INFINITY, cross = 0.f;
  if constexpr (DENSE) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = l[v] == l[v] ? l[v] : -INFINITY;
      m = fmaxf(m, l[v]);
    }
    m = wave_max(m);
    float z = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = soft_num(l[v], m);
      z += l[v];
    }
    z = wave_sum(z);
    zi = z > 0 ? 1.f / z : 0.f;
    cross = wave_sum(soft_num(lj, m) * zi * g);
    val = g;
  } else if (p.softmax) {
    m = wave_max(lj);
    const float n = soft_num(lj, m);
    const float S = wave_sum(n);
    const float q = S > 0 ? n / S : 0.f;
    val = q * (g - wave_sum(q * g));
  } else {
    // in 64 bits, as the forward's: scores that fp32 cannot hold still have their shares
    const double s = sigmoid64(lj);
    const float s1 = 1.f / (1.f + expf(lj));  // 1 - s without its loss
    if (p.renorm) {
      const double S = wave_sum(s);
      const float q = S > 0 ? (float)(s / S) : 0.f;
      val = q * (g - wave_sum(g * q)) * s1;
    } else {
      val = g * (float)s * s1;
    }
  }
  float* mine = rows[wave];
  int* marks = reinterpret_cast<int*>(mine);
  if (e >= 0) marks[e] = lane;
  __syncthreads();
  const bool twice = __any(e >= 0 && marks[e] != lane);
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) mine[v * kWave + lane] = 0.f;
  __syncthreads();
  if (!twice) {
    if (e >= 0) mine[e] = val;
  } else {
    for (int j = 0; j < k; ++j)
      if (lane == j && e >= 0) mine[e] += val;
  }
  __syncthreads();
  if (!live) return;
  auto final = [&](int v, float a) { return DENSE ? l[v] * zi * (a - cross) : a; };
  if (V >= 4 && vec) {
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      if (e0 + v >= E) break;
      f32x4 x = *reinterpret_cast<const f32x4*>(mine + e0 + v);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = final(v + i < V ? v + i : 0, x[i]);
      f32x4* o = reinterpret_cast<f32x4*>(out + e0 + v);
      if (accumulate) {
        const f32x4 q = *o;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = add_rounded(q[i], x[i]);
      }
      *o = x;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (e0 + v >= E) break;
      const float x = final(v, mine[e0 + v]);
      out[e0 + v] = accumulate ? add_rounded(out[e0 + v], x) : x;
    }
  }
}

// Calls f with the experts a lane holds as a constant: the least power of two that covers E.
template <class Fn>
void with_experts(int E, Fn&& f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}
// Whether every row of [T, E] fp32 starts on a 16-byte boundary and holds whole pieces.
int whole_pieces(const void* p, int E) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && E % 4 == 0;
}

}  // namespace

hipError_t launch_gate_select(const GateParams& p, const float* logits, const float* bias, int T,
                              int E, int k, int32_t* idx, float* w, hipStream_t s) {
  // The definition compares scores under sums of two, also where every group stays and no sum is
  // needed: scores that meet in 64 bits (saturated sigmoids) are ties, their logits are not.
  const bool by_logit = !bias && (p.groups == 1 || !p.top2);
  const int vec = whole_pieces(logits, E);
  const dim3 grid((T + kGateWaves - 1) / kGateWaves), block(kGateWaves * kWave);
  {
    TraceScope trace("gate_select", s);
    with_experts(E, [&](auto v) {
      constexpr int V = decltype(v)::value;
      // the groups' LDS, where they are not whole runs of lanes
      const int gs = E / p.groups, lpg = gs / V;
      const bool lds = p.groups > 1 && p.topk_groups < p.groups &&
                       (gs % V != 0 || (lpg & (lpg - 1)) != 0);
      const size_t bytes = lds ? kGateWaves * (E + p.groups) * sizeof(double) : 0;
      if (by_logit)
        hipLaunchKernelGGL((gate_select_kernel<V, true>), grid, block, bytes, s, p, logits, bias,
                           T, E, k, vec, idx, w);
      else
        hipLaunchKernelGGL((gate_select_kernel<V, false>), grid, block, bytes, s, p, logits, bias,
                           T, E, k, vec, idx, w);
    });
  }
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateParams& p, const float* logits, const int32_t* idx,
                                const float* dw, int T, int E, int k, float* dlogits,
                                int accumulate, hipStream_t s) {
  const int vec = whole_pieces(dlogits, E) && whole_pieces(logits, E);
  const dim3 grid((T + kGateWaves - 1) / kGateWaves), block(kGateWaves * kWave);
  {
    TraceScope trace("gate_backward", s);
    with_experts(E, [&](auto v) {
      constexpr int V = decltype(v)::value;
      if (p.softmax && !p.renorm)
        hipLaunchKernelGGL((gate_backward_kernel<V, true>), grid, block, 0, s, p, logits, idx, dw,
                           T, E, k, vec, dlogits, accumulate);
      else
        hipLaunchKernelGGL((gate_backward_kernel<V, false>), grid, block, 0, s, p, logits, idx, dw,
                           T, E, k, vec, dlogits, accumulate);
    });
  }
  return hipGetLastError();
}

}  // namespace moe
