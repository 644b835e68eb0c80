// Internal launch interface of the gate, the router gradients, the block-scaled FP8 and int8
// products and the dense feed-forward block
// (kernels.h holds the layer's own). Every function only enqueues on the given stream and
// returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// gate.hip
struct GateParams {
  int softmax;      // scores: softmax over the row, else a sigmoid of each logit
  int groups;       // the E experts in this many equal runs
  int topk_groups;  // groups a token may choose from
  int top2;         // a group's score: the sum of its two largest choice scores, else its largest
  int renorm;       // weights divided by their sum over the selected
  float scale;      // and multiplied by this
};
hipError_t launch_gate_select(const GateParams& p, const float* logits, const float* bias, int T,
                              int E, int k, int32_t* idx, float* w, hipStream_t s);
hipError_t launch_gate_backward(const GateParams& p, const float* logits, const int32_t* idx,
                                const float* dw, int T, int E, int k, float* dlogits,
                                int accumulate, hipStream_t s);

// router_grad.hip
struct RouterGradArgs {
  const uint16_t* x;   // bf16 [T, d]
  const uint16_t* wr;  // bf16 [E, d]
  const float* dl;     // fp32 [T, E]
  uint16_t* dx;        // bf16 [T, d]
  float* dwr;          // fp32 [E, d]
  int T, d, E, acc_dx, acc_dwr;
};
hipError_t launch_router_backward(const RouterGradArgs& a, hipStream_t s);

// fp8.hip: E4M3 codes with one fp32 scale per block of 128 (rows) or 128 x 128 (weights)
hipError_t launch_fp8_quant_rows(const uint16_t* src, int rows, int cols, uint8_t* codes,
                                 float* scales, hipStream_t s);
hipError_t launch_fp8_quant_weights(const uint16_t* src, int E, int N, int K, uint8_t* codes,
                                    float* scales, uint8_t* codes_t, float* scales_t,
                                    hipStream_t s);
// The FP8 mode's steps around its products; M rows in position order, `placed` (device) of them
// in use. Scales are [columns / 128, M].
hipError_t launch_fp8_quant_gather(const uint16_t* src, const int32_t* row_src, int k,
                                   const int32_t* placed, int M, int cols, uint8_t* codes,
                                   float* scales, hipStream_t s);
hipError_t launch_fp8_swiglu(const uint16_t* H, const int32_t* placed, int M, int I, uint16_t* A,
                             uint8_t* codes, float* scales, hipStream_t s);
struct Fp8SwigluBwdArgs {
  const uint16_t* dAp;     // bf16 [M, I]
  const uint16_t* H;       // bf16 [M, 2I]
  const uint16_t* A;       // bf16 [M, I]
  const int32_t* row_src;  // [M]
  const float* topk_w;     // [M] flat
  const int32_t* placed;
  int M, I;
  uint16_t* dH;            // bf16 [M, 2I]
  uint8_t* codes;          // dH's codes [M, 2I]
  float* scales;
  float* dwpart;           // [M, I / 128]
};
hipError_t launch_fp8_swiglu_bwd(const Fp8SwigluBwdArgs& a, hipStream_t s);

struct Fp8GemmArgs {
  const int32_t* offsets;  // [E + 1]
  const uint8_t* a;        // [M, K] codes
  const float* sa;         // [K / 128, M]
  const uint8_t* b;        // [E, N, K] codes
  const float* sb;         // [E, N / 128, K / 128]
  uint16_t* out;           // [M, N] bf16
  int M, E, N, K;
};
hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t s);

// int8.hip: int8 codes with one fp32 scale a row (tokens) or output channel (weights)
hipError_t launch_i8_quant_rows(const uint16_t* src, long long rows, int cols, uint8_t* codes,
                                float* scales, hipStream_t s);
struct I8GemmArgs {
  const int32_t* offsets;  // [E + 1]
  const uint8_t* a;        // [M, K] codes
  const float* sa;         // [M]
  const uint8_t* b;        // [E, N, K] codes; gated: N = 2I, gate rows then up rows
  const float* sb;         // [E, N]
  uint16_t* out;           // [M, N] bf16; gated [M, N / 2]
  int M, E, N, K, act;
};
hipError_t launch_i8_gemm(const I8GemmArgs& a, bool gated, hipStream_t s);

// ffn.hip: the dense gated feed-forward block, bf16
struct FfnArgs {
  const uint16_t* x;   // [T, d]
  const uint16_t* w1;  // [2I, d]
  const uint16_t* w2;  // [d, I]
  uint16_t* H;         // [T, 2I]; the forward's may be null
  uint16_t* A;         // [T, I]
  uint16_t* y;         // [T, d]
  const uint16_t* dy;  // [T, d]
  uint16_t* dH;        // [T, 2I]
  uint16_t* dx;        // [T, d]
  float* part;         // sums of products split along K, kFfnPartBytes
  int T, d, I, act, acc_y, acc_dx, shares;
};
constexpr size_t kFfnPartBytes = size_t(256) * 128 * 128 * 4;  // a 128 x 128 tile a CU
struct FfnDwArgs {
  const uint16_t* L;  // [T, Md]
  const uint16_t* R;  // [T, Nd]
  void* dw;           // [Md, Nd] fp32, or (bf16_dw) bf16
  float* part;        // as in FfnArgs
  int T, Md, Nd, acc, bf16_dw, shares;
};
hipError_t launch_ffn_gate_up(const FfnArgs& a, hipStream_t s);
hipError_t launch_ffn_down(const FfnArgs& a, hipStream_t s);
// Each: a gradient of rows and one of weights
hipError_t launch_ffn_dh_dw2(const FfnArgs& a, const FfnDwArgs& dw, hipStream_t s);
hipError_t launch_ffn_dx_dw1(const FfnArgs& a, const FfnDwArgs& dw, hipStream_t s);

}  // namespace moe
