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
#include "common.h"
#include "kernels.h"
#include "ops.h"

namespace moe {
namespace {

constexpr int kGateMaxE = 1024;
constexpr int kGateQ = kGateMaxE / kWave;
constexpr int kGateWaves = 4;

MOE_DEV float wave_max(float v) {
#pragma unroll
  for (int o = kWave / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
template <class F>
MOE_DEV F wave_sum(F v) {
#pragma unroll
  for (int o = kWave / 2; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Softmax numerator of logit l under the row's largest m: 1 at the largest (so +inf entries
// share the row), 0 for a closed expert and in a row that holds nothing else.
template <class F>
MOE_DEV F soft_num(float l, float m) {
  if (l == -INFINITY) return F(0);
  if (l == m) return F(1);
  return exp(F(l) - F(m));
}

// One wave per token; choice scores and group scores in LDS.
__global__ void __launch_bounds__(kGateWaves* kWave) gate_select_kernel(
    GateParams p, const float* __restrict__ logits, const float* __restrict__ bias, int T, int E,
    int k, int32_t* __restrict__ idx, float* __restrict__ w) {
  extern __shared__ double gate_lds[];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int t = blockIdx.x * kGateWaves + wave;
  const bool live = t < T;
  const int G = p.groups, gs = E / G;
  double* cs = gate_lds + (size_t)wave * (E + G);
  double* gsc = cs + E;
  const float* row = logits + (size_t)(live ? t : 0) * E;
  const bool by_logit = !bias && (G == 1 || !p.top2);
  float l[kGateQ];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < kGateQ; ++q) {
    const int e = lane + kWave * q;
    float v = e < E ? row[e] : -INFINITY;
    l[q] = v == v ? v : -INFINITY;
    m = fmaxf(m, l[q]);
  }
  m = wave_max(m);
  double sc[kGateQ], z = 0;
#pragma unroll
  for (int q = 0; q < kGateQ; ++q) {
    if (p.softmax) {
      sc[q] = soft_num<double>(l[q], m);
      z += sc[q];
    } else {
      sc[q] = l[q] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)l[q]));
    }
  }
  if (p.softmax) {
    z = wave_sum(z);
#pragma unroll
    for (int q = 0; q < kGateQ; ++q) sc[q] = z > 0 ? sc[q] / z : 0.0;
  }
  double c[kGateQ];
#pragma unroll
  for (int q = 0; q < kGateQ; ++q) {
    const int e = lane + kWave * q;
    c[q] = l[q] == -INFINITY ? -INFINITY
           : by_logit        ? (double)l[q]
                             : sc[q] + (bias ? (double)bias[e < E ? e : 0] : 0.0);
    if (e < E) cs[e] = c[q];
  }
  __syncthreads();
  for (int g = lane; g < G; g += kWave) {
    double a = -INFINITY, b = -INFINITY;
    for (int i = 0; i < gs; ++i) {
      const double v = cs[g * gs + i];
      if (v > a) {
        b = a;
        a = v;
      } else if (v > b) {
        b = v;
      }
    }
    gsc[g] = p.top2 && b != -INFINITY ? a + b : a;
  }
  __syncthreads();
  // rounds of an argmax over the wave, the lower index first among equals
  auto best = [&](double bv, int be) {
#pragma unroll
    for (int o = kWave / 2; o; o >>= 1) {
      const double ov = __shfl_xor(bv, o);
      const int oe = __shfl_xor(be, o);
      if (oe >= 0 && (be < 0 || ov > bv || (ov == bv && oe < be))) {
        bv = ov;
        be = oe;
      }
    }
    return be;
  };
  uint32_t taken = 0;  // bit q: expert lane + 64 q selected or out of reach
  if (G > 1 && p.topk_groups < G) {
    uint32_t gt = 0;  // bit i: group lane + 64 i selected
    for (int r = 0; r < p.topk_groups; ++r) {
      double bv = -INFINITY;
      int be = -1;
      for (int i = 0; lane + kWave * i < G; ++i) {
        const double v = gsc[lane + kWave * i];
        if (!((gt >> i) & 1u) && (be < 0 || v > bv)) {
          bv = v;
          be = lane + kWave * i;
        }
      }
      be = best(bv, be);
      if (be % kWave == lane) gt |= 1u << (be / kWave);
    }
    __syncthreads();
    for (int i = 0; lane + kWave * i < G; ++i) gsc[lane + kWave * i] = (gt >> i) & 1u ? 1.0 : 0.0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kGateQ; ++q) {
      const int e = lane + kWave * q;
      if (e < E && gsc[e / gs] == 0.0) taken |= 1u << q;
    }
  }
  double mine = 0;
  int my_e = 0;
  for (int j = 0; j < k; ++j) {
    double bv = -INFINITY;
    int be = -1;
#pragma unroll
    for (int q = 0; q < kGateQ; ++q) {
      const int e = lane + kWave * q;
      if (e < E && !((taken >> q) & 1u) && (be < 0 || c[q] > bv)) {
        bv = c[q];
        be = e;
      }
    }
    be = best(bv, be);
    double s = 0;
#pragma unroll
    for (int q = 0; q < kGateQ; ++q)
      if (lane + kWave * q == be) {
        s = sc[q];
        taken |= 1u << q;
      }
    s = __shfl(s, be % kWave);
    if (lane == j) {
      mine = s;
      my_e = be;
    }
  }
  double sum = 0;
  for (int j = 0; j < k; ++j) sum += __shfl(mine, j);
  if (live && lane < k) {
    double v = mine;
    if (p.renorm) v = sum > 0 ? v / sum : 0.0;
    idx[(size_t)t * k + lane] = my_e;
    w[(size_t)t * k + lane] = (float)(v * (double)p.scale);
  }
}

// One wave per token. Lane j < k takes slot j, then every lane writes its logits' gradients.
//   g_j = scale dw_j
//   sigmoid:                 dl_j = g_j s_j (1 - s_j)
//   sigmoid, renormalised:   dl_j = (g_j - sum_i g_i q_i) / S  s_j (1 - s_j),  q = s / S
//   softmax, renormalised:   dl_j = q_j (g_j - sum_i q_i g_i)
//   softmax:                 dl_e = p_e ([e selected] g_e - sum_i p_i g_i), for every e
// Slots that name one expert twice add up, in ascending j; a slot outside [0, E) counts nothing.
__global__ void __launch_bounds__(kGateWaves* kWave) gate_backward_kernel(
    GateParams p, const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const float* __restrict__ dw, int T, int E, int k, float* __restrict__ dl, int accumulate) {
  const int lane = threadIdx.x % kWave;
  const int t = blockIdx.x * kGateWaves + threadIdx.x / kWave;
  if (t >= T) return;  // whole waves leave; no barrier below
  const float* row = logits + (size_t)t * E;
  float* out = dl + (size_t)t * E;
  int e = lane < k ? idx[(size_t)t * k + lane] : -1;
  if (e < 0 || e >= E) e = -1;
  float lj = e >= 0 ? row[e] : -INFINITY;
  if (!(lj == lj)) lj = -INFINITY;
  const float g = e >= 0 ? p.scale * dw[(size_t)t * k + lane] : 0.f;
  const bool dense = p.softmax && !p.renorm;
  float m = -INFINITY, z = 0.f, v = 0.f, cross = 0.f;
  if (dense) {
    for (int i = lane; i < E; i += kWave) m = fmaxf(m, row[i]);  // fmaxf drops a NaN
    m = wave_max(m);
    for (int i = lane; i < E; i += kWave) {
      const float x = row[i];
      if (x == x) z += soft_num<float>(x, m);
    }
    z = wave_sum(z);
    z = z > 0 ? 1.f / z : 0.f;
    cross = wave_sum(soft_num<float>(lj, m) * z * g);
    v = g;
  } else if (p.softmax) {
    m = wave_max(lj);
    const float n = soft_num<float>(lj, m);
    const float S = wave_sum(n);
    const float q = S > 0 ? n / S : 0.f;
    v = q * (g - wave_sum(q * g));
  } else {
    const float s = lj == -INFINITY ? 0.f : 1.f / (1.f + expf(-lj));
    const float s1 = lj == -INFINITY ? 0.f : 1.f / (1.f + expf(lj));  // 1 - s without its loss
    float ds = g;
    if (p.renorm) {
      const float S = wave_sum(s);
      ds = S > 0 ? (g - wave_sum(g * (s / S))) / S : 0.f;
    }
    v = ds * s * s1;
  }
  for (int i = lane; i < E; i += kWave) {
    float a = 0.f;
    for (int j = 0; j < k; ++j) {
      const int ej = __builtin_amdgcn_readlane(e, j);
      const float vj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), j));
      if (ej == i) a += vj;
    }
    if (dense) {
      const float x = row[i];
      a = x == x ? soft_num<float>(x, m) * z * (a - cross) : 0.f;
    }
    out[i] = accumulate ? out[i] + a : a;
  }
}

}  // namespace

hipError_t launch_gate_select(const GateParams& p, const float* logits, const float* bias, int T,
                              int E, int k, int32_t* idx, float* w, hipStream_t s) {
  {
    TraceScope trace("gate_select", s);
    hipLaunchKernelGGL(gate_select_kernel, dim3((T + kGateWaves - 1) / kGateWaves),
                       dim3(kGateWaves * kWave), kGateWaves * (E + p.groups) * sizeof(double), s,
                       p, logits, bias, T, E, k, idx, w);
  }
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateParams& p, const float* logits, const int32_t* idx,
                                const float* dw, int T, int E, int k, float* dlogits,
                                int accumulate, hipStream_t s) {
  {
    TraceScope trace("gate_backward", s);
    hipLaunchKernelGGL(gate_backward_kernel, dim3((T + kGateWaves - 1) / kGateWaves),
                       dim3(kGateWaves * kWave), 0, s, p, logits, idx, dw, T, E, k, dlogits,
                       accumulate);
  }
  return hipGetLastError();
}

}  // namespace moe
