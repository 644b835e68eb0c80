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
// a in the lanes of the mask, b in the others. In assembly, since a chain of selects between
// neighbours of an array is otherwise turned into selects by an index, among all of them.
MOE_DEV uint32_t select_lanes(uint64_t mask, uint32_t a, uint32_t b) {
  asm("v_cndmask_b32_e64 %0, %1, %2, %3" : "=v"(b) : "0"(b), "v"(a), "s"(mask));
  return b;
}
MOE_DEV double select_lanes(uint64_t mask, double a, double b) {
  const uint64_t x = __builtin_bit_cast(uint64_t, a), y = __builtin_bit_cast(uint64_t, b);
  return __builtin_bit_cast(
      double, (uint64_t)select_lanes(mask, (uint32_t)x, (uint32_t)y) |
                  ((uint64_t)select_lanes(mask, (uint32_t)(x >> 32), (uint32_t)(y >> 32)) << 32));
}
MOE_DEV uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
MOE_DEV float larger(float a, float b) { return fmaxf(a, b); }
MOE_DEV double larger(double a, double b) { return __builtin_fmax(a, b); }
MOE_DEV uint32_t smaller(uint32_t a, uint32_t b) { return min(a, b); }
MOE_DEV double smaller(double a, double b) { return __builtin_fmin(a, b); }
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
// e^r by its Taylor polynomial of degree 12 (the next term is below 1.8e-16), about 1e-15 in
// all. 20 instructions; the library's exp also covers what does not occur here.
MOE_DEV double exp64(double x) {
  x = __builtin_fmax(x, -745.0);
  // adding 1.5 2^52 rounds to a whole number, which the sum's low word then holds
  const double t = __builtin_fma(x, 1.4426950408889634, 6755399441055744.0);
  const double n = t - 6755399441055744.0;
  double r = __builtin_fma(n, -6.93147180369123816490e-01, x);
  r = __builtin_fma(n, -1.90821492927058770002e-10, r);
  double p = 1.0 / 479001600.0;
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
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

// v[0] >= v[1] >= .., by merging sorted halves (odd-even merges: 1, 5, 19, 63 exchanges).
template <int V, class C>
MOE_DEV void sort_down(C (&v)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const C a = v[i + j], b = v[i + j + q];
            v[i + j] = larger(a, b);
            v[i + j + q] = smaller(a, b);
          }
}

// One wave per token: lane l holds the V experts from V l on, so that the lowest lane and then
// its lowest slot that hold a value hold the lowest index. Each lane sorts its V choice scores;
// k rounds then take the wave's largest head (DPP shifts, no LDS) from the lowest lane that has
// it. A round costs the same for any V but for the lane's V moves; which of its V experts a lane
// gave is worked out once, for all k choices together.
// LOGIT: the scores order as the logits do; 32-bit keys, and 64-bit scores only of the chosen.
// Groups that are whole, aligned runs of 2^i lanes are scored by lane exchanges, others in LDS.
// Measured on 2048 x 256 (8 groups, sigmoid, bias) and 18944 x 512 (softmax): see the launch.
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
      } else {  // a closed expert's 5e-324 does not change a sum that holds a 1
#pragma unroll
        for (int v = 0; v < V; ++v) z += exp64((double)l[v] - (double)m);
      }
      z = wave_sum(z);
      zi = m > -INFINITY ? rcp64(z) : 0.0;
    }
  }
  C c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (LOGIT) {
      c[v] = e0 + v < E ? order32(l[v]) : kTaken;
    } else {
      const double s = !p.softmax      ? sigmoid64(l[v])
                       : m == INFINITY ? (l[v] == INFINITY ? zi : 0.0)
                                       : exp64((double)l[v] - (double)m) * zi;
      const double x = s + (bias ? (double)bias[min(e0 + v, E - 1)] : 0.0);
      c[v] = e0 + v >= E ? kTaken : l[v] > -INFINITY && x > kClosed ? x : kClosed;
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
      for (int o = 1; o < lpg; o <<= 1) {
        const C a1 = __shfl_xor(a, o), b1 = __shfl_xor(b, o);
        const C lo = a1 > a ? a : a1;
        a = larger(a, a1);
        b = larger(larger(b, b1), lo);
      }
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
        if (e0 + v < E && gsc[(e0 + v) / gs] == 0.0) c[v] = kTaken;
    }
  }
  // rounds: the wave's largest head, from the lowest lane that has it
  C h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = c[v];
  sort_down(h);
  C my_c = kTaken, last = kTaken;
  int my_at = 0, owner = -1, occ = 0;  // lane j: owner | occ << 8 of choice j
  for (int j = 0; j < k; ++j) {
    const C top = wave_max(h[0]);
    const int o = __builtin_ctzll(__ballot(h[0] == top));
    occ = o == owner && top == last ? occ + 1 : 0;  // the same value again in the same lane
    owner = o;
    last = top;
    const uint64_t pop = 1ull << o, mine = 1ull << j;
    my_c = select_lanes(mine, top, my_c);
    my_at = (int)select_lanes(mine, (uint32_t)(o | occ << 8), (uint32_t)my_at);
#pragma unroll
    for (int v = 0; v + 1 < V; ++v) h[v] = select_lanes(pop, h[v + 1], h[v]);
    h[V - 1] = lane == o ? kTaken : h[V - 1];
  }
  // lane j finds its expert: the occ-th of the owner's values that equal its own
  int my_e = 0;
  {
    const int o = my_at & 0xff;
    const int skip = my_at >> 8;
    int at = 0;
    int seen = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool hit = __shfl(c[v], o) == my_c;
      at = hit && seen == skip ? v : at;
      seen += hit;
    }
    my_e = o * V + at;
  }
  float my_l;
  if constexpr (LOGIT) my_l = unorder32(my_c);
  else my_l = lane < k ? row[my_e] : -INFINITY;
  my_l = my_l == my_l ? my_l : -INFINITY;
  double s = 0;  // lane j: the score of choice j
  if (lane < k) {
    s = !p.softmax ? sigmoid64(my_l) : soft_num64(my_l, m);
    if (p.softmax && zi > 0) s *= zi;
  }
  if (p.renorm) {
    const double sum = wave_sum(s);
    s = sum > 0 ? s / sum : 0.0;
  } else if (p.softmax && !(zi > 0)) {
    s = 0;
  }
  if (live && lane < k) {
    idx[(size_t)t * k + lane] = my_e;
    w[(size_t)t * k + lane] = (float)(s * (double)p.scale);
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
  const bool by_logit = !bias && (p.groups == 1 || p.topk_groups == p.groups || !p.top2);
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
