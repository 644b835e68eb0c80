// C ABI of the MoE layer: argument checks, buffer layout and launch sequences.
// Every call checks its arguments on the host, then enqueues its kernels on the caller's
// stream. It never allocates, synchronises or prints.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "moe.h"
#include "kernels.h"
#include "ops.h"

namespace {

using namespace moe;
static_assert(MOE_STATIC_SCRATCH_BYTES == kStaticPermScratchBytes, "one size in both places");

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

struct Layout {
  bool mx, f8, i8;  // the MX modes; the block-scaled FP8 mode; the INT8 mode
  int fb;  // MX code bits: 8 (MXFP8) or 4 (MXFP4); 0 in BF16 mode
  // workspace
  size_t status, sched, blk_cnt, blk_flag, rank, O, dH, dXp, dyw, dwpart, dl_pos, wg_count,
      wg_table1, wg_table2, wr32, total;
  // workspace, MX modes only: dY, A and dH quantised along their GEMM's K (codes, scales)
  size_t dyq, dys, aq, aqs, dhq, dhs;
  // workspace, MXFP8 weight gradients only: padded segment offsets [E + 1], and the two
  // operands of one weight gradient quantised along the positions, [rows][P] with scales
  size_t poff, lq, lqs, rq, rqs;
  int P;
  // workspace, FP8 mode only: the rows of one product quantised (Xp, A, dY or dH), and dA'
  size_t f8q, f8s, dAp;
  // workspace, INT8 mode only: the rows of one product quantised (Xp or A)
  size_t i8q, i8s;
  // saved
  size_t H, A, saved_total;
  // ring slot: bf16 Xp, or MX Xp codes at 0 and scales at slot_sc
  size_t slot, slot_sc;
  // quantised weights (MX): W1 and W2 along their forward K, and transposed along their
  // dgrad K: W1f [E,2I,d], W2f [E,d,I], W2b [E,I,d], W1b [E,d,2I], each with per-32 scales
  size_t w1f, w1fs, w2f, w2fs, w2b, w2bs, w1b, w1bs, wq_total;
  int nb, nIt, max_mtiles;
};

bool cfg_ok(const moe_cfg* c) {
  if (!c) return false;
  if (c->T < 1 || c->d < 256 || c->d % 256 != 0 || c->I < 128 || c->I % 128 != 0) return false;
  if (c->E < 1 || c->E > 1024 || c->k < 1 || c->k > c->E || c->k > kMaxTopK) return false;
  const long long T = c->T, d = c->d, I = c->I, Tk = T * c->k;
  if (Tk >= (1LL << 31) || T * c->E >= (1LL << 31)) return false;
  // The kernels address rows with 32-bit offsets. Element offsets into X and dY, and byte
  // offsets into one expert's rows of Xp, dXp, dYw, H, A and dH: a caller's routing may send
  // every row to one expert (a token may even repeat an expert), so an expert has up to T*k
  // rows. Byte offsets into one expert's weights: W1[e] is 2I x d bf16.
  if (T * d >= (1LL << 31)) return false;
  if (Tk * d >= (1LL << 31) || Tk * 2 * I >= (1LL << 31)) return false;
  if (4 * I * d >= (1LL << 31)) return false;
  return true;
}

// The kernels are built for gfx950 only. The current device's architecture is read once per
// device and kept.
int check_device() {
  constexpr int kMaxDev = 64;
  static std::atomic<int> arch_seen[kMaxDev];  // 0 unknown, 1 gfx950, 2 another device
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return MOE_ERR_HIP;
  }
  if (dev < kMaxDev) {
    const int v = arch_seen[dev].load(std::memory_order_relaxed);
    if (v) return v == 1 ? MOE_OK : MOE_ERR_UNSUPPORTED;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ERR_HIP;
  }
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 &&
                  (prop.gcnArchName[6] == 0 || prop.gcnArchName[6] == ':');
  if (dev < kMaxDev) arch_seen[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

Layout layout(const moe_cfg* c) {
  Layout L{};
  const size_t Tk = (size_t)c->T * c->k, d = c->d, I = c->I, E = c->E;
  L.nb = (int)((Tk + kPermRows - 1) / kPermRows);
  L.nIt = c->I / kDgradBN;
  L.max_mtiles = sched_max_mtiles((int)Tk, c->E);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  L.status = take(16);
  L.sched = take(sizeof(int2) * sched_entries((int)Tk, (int)E));
  L.blk_cnt = take(sizeof(int32_t) * (size_t)L.nb * E);
  L.blk_flag = take(sizeof(int32_t) * (size_t)L.nb);
  L.rank = take(sizeof(int32_t) * Tk);
  L.O = take(2 * Tk * d);
  L.dH = take(2 * Tk * 2 * I);
  L.dXp = take(2 * Tk * d);
  L.dyw = take(2 * Tk * d);
  L.wg_count = take(2 * sizeof(int32_t));
  L.wg_table1 = take(16 * wgrad_table_entries((int)Tk, c->E, 2 * c->I, c->d));
  L.wg_table2 = take(16 * wgrad_table_entries((int)Tk, c->E, c->d, c->I));
  L.dwpart = take(sizeof(float) * Tk * L.nIt);
  L.dl_pos = take(sizeof(float) * Tk);
  L.wr32 = take(sizeof(float) * E * d);
  L.mx = c->precision == MOE_PREC_MXFP8 || c->precision == MOE_PREC_MXFP4;
  L.fb = c->precision == MOE_PREC_MXFP8 ? 8 : c->precision == MOE_PREC_MXFP4 ? 4 : 0;
  const size_t T = c->T, mxs = L.mx ? 1 : 0;
  // bytes of n codes
  auto cb = [&](size_t n) { return n * L.fb / 8; };
  L.dyq = take(mxs * cb(T * d));
  L.dys = take(mxs * T * d / 32);
  L.aq = take(mxs * cb(Tk * I));
  L.aqs = take(mxs * Tk * I / 32);
  L.dhq = take(mxs * cb(Tk * 2 * I));
  L.dhs = take(mxs * Tk * 2 * I / 32);
  const size_t mxw = L.mx && (c->flags & MOE_FLAG_MXFP8_WGRAD) ? 1 : 0;
  L.P = mxw ? seg_capacity((int)Tk, c->E) : 0;
  const size_t P = L.P, lrows = std::max(2 * I, d), rrows = std::max(d, I);
  L.poff = take(mxw * sizeof(int32_t) * (E + 1));
  L.lq = take(lrows * P);
  L.lqs = take(lrows * P / 32);
  L.rq = take(rrows * P);
  L.rqs = take(rrows * P / 32);
  L.f8 = c->precision == MOE_PREC_FP8;
  const size_t f8 = L.f8 ? 1 : 0, fcols = std::max(d, 2 * I);
  L.f8q = take(f8 * Tk * fcols);
  L.f8s = take(f8 * sizeof(float) * Tk * (fcols / 128));
  L.dAp = take(f8 * 2 * Tk * I);
  L.i8 = c->precision == MOE_PREC_INT8;
  const size_t i8 = L.i8 ? 1 : 0;
  L.i8q = take(i8 * Tk * std::max(d, I));
  L.i8s = take(i8 * sizeof(float) * Tk);
  L.total = o;
  o = 0;
  L.H = take(L.i8 ? 0 : 2 * Tk * 2 * I);
  L.A = take(2 * Tk * I);
  L.saved_total = o;
  if (L.mx) {
    o = 0;
    take(cb(Tk * d));
    L.slot_sc = o;
    take(Tk * d / 32);
    L.slot = o;
    o = 0;
    L.w1f = take(cb(E * 2 * I * d));
    L.w1fs = take(E * 2 * I * d / 32);
    L.w2f = take(cb(E * d * I));
    L.w2fs = take(E * d * I / 32);
    L.w2b = take(cb(E * I * d));
    L.w2bs = take(E * I * d / 32);
    L.w1b = take(cb(E * d * 2 * I));
    L.w1bs = take(E * d * 2 * I / 32);
    L.wq_total = o;
  } else {
    L.slot = 2 * Tk * d;
  }
  if (L.f8) {  // both orientations of both weights, a scale per 128 x 128
    const size_t n1 = E * 2 * I * d, n2 = E * d * I;
    o = 0;
    L.w1f = take(n1);
    L.w1fs = take(sizeof(float) * (n1 / 16384));
    L.w2f = take(n2);
    L.w2fs = take(sizeof(float) * (n2 / 16384));
    L.w2b = take(n2);
    L.w2bs = take(sizeof(float) * (n2 / 16384));
    L.w1b = take(n1);
    L.w1bs = take(sizeof(float) * (n1 / 16384));
    L.wq_total = o;
  }
  if (L.i8) {  // the forward's weights, a scale per output channel
    o = 0;
    L.w1f = take(E * 2 * I * d);
    L.w1fs = take(sizeof(float) * E * 2 * I);
    L.w2f = take(E * d * I);
    L.w2fs = take(sizeof(float) * E * d);
    L.wq_total = o;
  }
  return L;
}

bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) % 16) == 0; }
bool aligned4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) % 4) == 0; }

template <class T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}
template <class T>
const T* at(const void* base, size_t off) {
  return reinterpret_cast<const T*>(static_cast<const char*>(base) + off);
}

// First error wins; later launches are skipped once one fails.
struct Launches {
  hipError_t err = hipSuccess;
  void operator()(hipError_t e) {
    if (err == hipSuccess) err = e;
  }
  int status() const { return err == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
};

int check_mode(const moe_cfg* c) {
  if (!cfg_ok(c)) return MOE_ERR_INVALID_ARG;
  if (c->precision != MOE_PREC_BF16 && c->precision != MOE_PREC_MXFP8 &&
      c->precision != MOE_PREC_MXFP4 && c->precision != MOE_PREC_FP8 &&
      c->precision != MOE_PREC_INT8)
    return MOE_ERR_UNSUPPORTED;
  if (c->precision == MOE_PREC_INT8) {
    const long long top = 1LL << 24, E = c->E;  // rows of one quantisation
    if (c->flags || c->d >= (1 << 17) || c->I >= (1 << 17) || (long long)c->T * c->k >= top ||
        E * 2 * c->I >= top || E * c->d >= top)
      return MOE_ERR_INVALID_ARG;
  }
  if (c->precision == MOE_PREC_FP8 && (c->flags & MOE_FLAG_PERSISTENT)) return MOE_ERR_INVALID_ARG;
  if (c->precision == MOE_PREC_MXFP4 && c->I % 256 != 0) return MOE_ERR_INVALID_ARG;
  if (c->flags & ~(MOE_FLAG_PERSISTENT | MOE_FLAG_MXFP8_WGRAD | MOE_FLAG_BF16_DW))
    return MOE_ERR_INVALID_ARG;
  if ((c->flags & MOE_FLAG_MXFP8_WGRAD) && c->precision != MOE_PREC_MXFP8)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_ring(const Layout& L, const void* ring, size_t ring_bytes, int32_t slot) {
  if (!aligned16(ring)) return MOE_ERR_INVALID_ARG;
  if (slot < 0 || (size_t)(slot + 1) * L.slot > ring_bytes) return MOE_ERR_RING_TOO_SMALL;
  return MOE_OK;
}

// The quantised weights of the MX modes, or an error code when they are missing.
int check_wq(const Layout& Y, const void* wq, size_t wq_bytes) {
  if (!Y.mx && !Y.f8 && !Y.i8) return MOE_OK;
  if (!aligned16(wq)) return MOE_ERR_INVALID_ARG;
  if (wq_bytes < Y.wq_total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return MOE_OK;
}

int check_gate(const moe_cfg* c, const moe_gate* g) {
  if (!g) return MOE_ERR_INVALID_ARG;
  if (g->score != MOE_SCORE_SOFTMAX && g->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (g->group_score != MOE_GROUP_MAX && g->group_score != MOE_GROUP_TOP2)
    return MOE_ERR_INVALID_ARG;
  if (g->groups < 1 || g->groups > c->E || c->E % g->groups != 0) return MOE_ERR_INVALID_ARG;
  if (g->topk_groups < 1 || g->topk_groups > g->groups) return MOE_ERR_INVALID_ARG;
  if (c->k > g->topk_groups * (c->E / g->groups)) return MOE_ERR_INVALID_ARG;
  if ((g->renorm != 0 && g->renorm != 1) || !std::isfinite(g->scale)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Weights [E, N, K] of the block-scaled FP8 calls.
int check_fp8_shape(int32_t E, int32_t N, int32_t K) {
  if (E < 1 || E > 1024 || N < 128 || N % 128 != 0 || K < 128 || K % 128 != 0 ||
      (long long)N * K >= (1LL << 31))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_i8_shape(int32_t E, int32_t N, int32_t K) {
  if (const int st = check_fp8_shape(E, N, K)) return st;
  return K < (1 << 17) ? MOE_OK : MOE_ERR_INVALID_ARG;  // 128 * 128 * K stays below 2^31
}

bool act_ok(int32_t act) { return act >= MOE_ACT_SILU && act <= MOE_ACT_RELU; }

int i8_gemm(const int32_t* offsets, int32_t M, int32_t E, int32_t N, int32_t K, int32_t act,
            bool gated, const void* a, const float* a_scales, const void* b,
            const float* b_scales, void* out, moe_stream_t stream) {
  if (const int st = check_i8_shape(E, N, K)) return st;
  if (M < 0 || !aligned4(offsets) || !aligned16(b) || !aligned4(b_scales))
    return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;  // empty buffers have no address to check
  if (!aligned16(a) || !aligned4(a_scales) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  // every kernel's grid has fewer than 2^32 threads
  if ((M / 128LL + 2 * E) * (N / 128) >= (1LL << 24)) return MOE_ERR_INVALID_ARG;
  if (const int st = check_device()) return st;
  I8GemmArgs g{offsets, static_cast<const uint8_t*>(a), a_scales, static_cast<const uint8_t*>(b),
               b_scales, static_cast<uint16_t*>(out), M, E, N, K, act};
  Launches L;
  L(launch_i8_gemm(g, gated, static_cast<hipStream_t>(stream)));
  return L.status();
}

int check_ffn(const moe_ffn* f) {
  if (!f || f->T < 1 || f->d < 128 || f->d % 128 != 0 || f->I < 128 || f->I % 128 != 0 ||
      !act_ok(f->act) || (f->flags & ~MOE_FLAG_BF16_DW))
    return MOE_ERR_INVALID_ARG;
  const long long T = f->T, d = f->d, I = f->I;
  if ((T + 64) * std::max(d, 2 * I) >= (1LL << 31) || 4 * I * d >= (1LL << 31))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
struct FfnLayout {
  size_t dH, part, part_dw, total;
};
FfnLayout ffn_layout(const moe_ffn* f) {
  FfnLayout L{};
  L.part = align_up(2 * (size_t)f->T * 2 * f->I);
  L.part_dw = L.part + kFfnPartBytes;
  L.total = L.part_dw + kFfnPartBytes;
  return L;
}

GateParams gate_params(const moe_gate* g) {
  GateParams p;
  p.softmax = g->score == MOE_SCORE_SOFTMAX;
  p.groups = g->groups;
  p.topk_groups = g->topk_groups;
  p.top2 = g->group_score == MOE_GROUP_TOP2;
  p.renorm = g->renorm;
  p.scale = g->scale;
  return p;
}

// Launch tracing (moe_trace_begin / moe_trace_end).
std::atomic<void* const*> g_trace_events{nullptr};
std::mutex g_trace_mu;
const char** g_trace_names = nullptr;
int g_trace_cap = 0;
int g_trace_count = 0;

}  // namespace

namespace moe {
void trace_pre(const char* name, hipStream_t s) {
  if (!g_trace_events.load(std::memory_order_acquire)) return;
  std::lock_guard<std::mutex> lk(g_trace_mu);
  void* const* ev = g_trace_events.load(std::memory_order_relaxed);
  const int i = g_trace_count;
  if (ev && 2 * i + 1 < g_trace_cap) {
    (void)hipEventRecord(static_cast<hipEvent_t>(ev[2 * i]), s);
    if (g_trace_names) g_trace_names[i] = name;
  }
}
void trace_post(hipStream_t s) {
  if (!g_trace_events.load(std::memory_order_acquire)) return;
  std::lock_guard<std::mutex> lk(g_trace_mu);
  void* const* ev = g_trace_events.load(std::memory_order_relaxed);
  const int i = g_trace_count++;
  if (ev && 2 * i + 1 < g_trace_cap) (void)hipEventRecord(static_cast<hipEvent_t>(ev[2 * i + 1]), s);
}
}  // namespace moe

extern "C" {

int moe_trace_begin(void* const* events, int capacity, const char** names) {
  if (!events || capacity < 2) return MOE_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lk(g_trace_mu);
  g_trace_names = names;
  g_trace_cap = capacity;
  g_trace_count = 0;
  g_trace_events.store(events, std::memory_order_release);
  return MOE_OK;
}

int moe_trace_end(void) {
  std::lock_guard<std::mutex> lk(g_trace_mu);
  g_trace_events.store(nullptr, std::memory_order_release);
  const int n = g_trace_count;
  g_trace_count = 0;
  g_trace_cap = 0;
  g_trace_names = nullptr;
  return n;
}

int moe_query(const moe_cfg* cfg, moe_sizes* out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  if (const int st = check_mode(cfg)) return st;
  const Layout L = layout(cfg);
  out->ring_slot = L.slot;
  out->saved = L.saved_total;
  out->saved_H = L.H;
  out->saved_A = L.A;
  out->workspace = L.total;
  out->ws_O = L.O;
  out->ws_dH = L.dH;
  out->ws_dXp = L.dXp;
  out->wq = L.mx || L.f8 || L.i8 ? L.wq_total : 0;
  return MOE_OK;
}

int moe_quantize_weights(const moe_cfg* cfg, const void* w1, const void* w2, void* wq,
                         size_t wq_bytes, moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  const Layout Y = layout(cfg);
  if (!Y.mx && !Y.f8 && !Y.i8) return MOE_ERR_INVALID_ARG;
  if (!aligned16(w1) || !aligned16(w2) || !aligned16(wq)) return MOE_ERR_INVALID_ARG;
  if (wq_bytes < Y.wq_total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device())) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int E = cfg->E, d = cfg->d, I = cfg->I;
  const uint16_t* a1 = static_cast<const uint16_t*>(w1);
  const uint16_t* a2 = static_cast<const uint16_t*>(w2);
  Launches L;
  if (Y.i8) {
    L(launch_i8_quant_rows(a1, 2LL * E * I, d, at<uint8_t>(wq, Y.w1f), at<float>(wq, Y.w1fs), s));
    if (!L.err)
      L(launch_i8_quant_rows(a2, (long long)E * d, I, at<uint8_t>(wq, Y.w2f),
                             at<float>(wq, Y.w2fs), s));
    return L.status();
  }
  if (Y.f8) {
    L(launch_fp8_quant_weights(a1, E, 2 * I, d, at<uint8_t>(wq, Y.w1f), at<float>(wq, Y.w1fs),
                               at<uint8_t>(wq, Y.w1b), at<float>(wq, Y.w1bs), s));
    if (!L.err)
      L(launch_fp8_quant_weights(a2, E, d, I, at<uint8_t>(wq, Y.w2f), at<float>(wq, Y.w2fs),
                                 at<uint8_t>(wq, Y.w2b), at<float>(wq, Y.w2bs), s));
    return L.status();
  }
  L(launch_quant_weight(a1, E, 2 * I, d, at<uint8_t>(wq, Y.w1f), at<uint8_t>(wq, Y.w1fs),
                        at<uint8_t>(wq, Y.w1b), at<uint8_t>(wq, Y.w1bs), Y.fb, "quant_w1", s));
  if (!L.err)
    L(launch_quant_weight(a2, E, d, I, at<uint8_t>(wq, Y.w2f), at<uint8_t>(wq, Y.w2fs),
                          at<uint8_t>(wq, Y.w2b), at<uint8_t>(wq, Y.w2bs), Y.fb, "quant_w2", s));
  return L.status();
}

int moe_route(const moe_cfg* cfg, const void* x, const void* w_router, float* logits,
              int32_t* topk_idx, float* topk_w, void* workspace, size_t ws_bytes,
              moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  if (!aligned16(x) || !aligned16(w_router) || !aligned4(logits) || !aligned4(topk_idx) ||
      !aligned4(topk_w) || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  const Layout Y = layout(cfg);
  if (ws_bytes < Y.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device())) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Launches L;
  L(launch_router_logits(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w_router),
                         at<float>(workspace, Y.wr32), logits, cfg->T, cfg->d, cfg->E, s));
  if (L.err == hipSuccess)
    L(launch_router_topk(logits, cfg->T, cfg->E, cfg->k, topk_idx, topk_w, s));
  return L.status();
}

int moe_permute(const moe_cfg* cfg, const int32_t* topk_idx, const void* x, void* ring,
                size_t ring_bytes, int32_t slot, int32_t* counts, int32_t* offsets,
                int32_t* row_src, int32_t* tk_row, void* workspace, size_t ws_bytes,
                moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  const Layout Y = layout(cfg);
  if (!aligned4(topk_idx) || !aligned16(x) || !aligned4(counts) || !aligned4(offsets) ||
      !aligned4(row_src) || !aligned4(tk_row) || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ring(Y, ring, ring_bytes, slot))) return st;
  if (ws_bytes < Y.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device())) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int Tk = cfg->T * cfg->k;
  int32_t* blk = at<int32_t>(workspace, Y.blk_cnt);
  int32_t* flag = at<int32_t>(workspace, Y.blk_flag);
  int32_t* rank = at<int32_t>(workspace, Y.rank);
  uint8_t* slot_base = at<uint8_t>(ring, (size_t)slot * Y.slot);
  uint16_t* xp = Y.mx ? nullptr : reinterpret_cast<uint16_t*>(slot_base);
  uint8_t* xp8 = Y.mx ? slot_base : nullptr;
  uint8_t* xps = Y.mx ? slot_base + Y.slot_sc : nullptr;
  Launches L;
  L(launch_perm_hist(topk_idx, Tk, cfg->E, blk, rank, flag, s));
  if (!L.err)
    L(launch_perm_scan(blk, Y.nb, cfg->E, flag, counts, offsets, at<int32_t>(workspace, Y.status),
                       s));
  if (!L.err)
    L(launch_perm_place(topk_idx, rank, blk, Tk, cfg->E, cfg->k, row_src, tk_row,
                        static_cast<const uint16_t*>(x), xp, xp8, xps, cfg->d, Y.fb, s));
  return L.status();
}

int moe_permute_static(const moe_cfg* cfg, const int32_t* topk_idx, const void* x, void* ring,
                       size_t ring_bytes, int32_t slot, int32_t* counts, int32_t* offsets,
                       int32_t* row_src, int32_t* tk_row, int32_t* device_status,
                       moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  const Layout Y = layout(cfg);
  if (!aligned4(topk_idx) || !aligned16(x) || !aligned4(counts) || !aligned4(offsets) ||
      !aligned4(row_src) || !aligned4(tk_row) || !aligned4(device_status))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ring(Y, ring, ring_bytes, slot))) return st;
  // the permutation's scratch, packed from offset 0 of the fixed array
  const size_t Tk = (size_t)cfg->T * cfg->k;
  const size_t o_flag = align_up(sizeof(int32_t) * (size_t)Y.nb * cfg->E);
  const size_t o_rank = o_flag + align_up(sizeof(int32_t) * (size_t)Y.nb);
  if (o_rank + sizeof(int32_t) * Tk > MOE_STATIC_SCRATCH_BYTES)
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device())) return st;
  void* base = nullptr;
  if (static_perm_scratch(&base) != hipSuccess) {
    (void)hipGetLastError();
    return MOE_ERR_HIP;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* slot_base = at<uint8_t>(ring, (size_t)slot * Y.slot);
  uint16_t* xp = Y.mx ? nullptr : reinterpret_cast<uint16_t*>(slot_base);
  uint8_t* xp8 = Y.mx ? slot_base : nullptr;
  uint8_t* xps = Y.mx ? slot_base + Y.slot_sc : nullptr;
  int32_t* blk = at<int32_t>(base, 0);
  int32_t* flag = at<int32_t>(base, o_flag);
  int32_t* rank = at<int32_t>(base, o_rank);
  // every scratch word is written before it is read: nothing needs clearing
  Launches L;
  L(launch_perm_hist(topk_idx, (int)Tk, cfg->E, blk, rank, flag, s));
  if (!L.err)
    L(launch_perm_scan(blk, Y.nb, cfg->E, flag, counts, offsets, device_status, s));
  if (!L.err)
    L(launch_perm_place(topk_idx, rank, blk, (int)Tk, cfg->E, cfg->k, row_src, tk_row,
                        static_cast<const uint16_t*>(x), xp, xp8, xps, cfg->d, Y.fb, s));
  return L.status();
}

int moe_forward(const moe_cfg* cfg, const void* ring, size_t ring_bytes, int32_t slot,
                const int32_t* offsets, const int32_t* tk_row, const float* topk_w,
                const void* w1, const void* w2, const void* wq, size_t wq_bytes, void* y,
                void* saved, size_t saved_bytes, void* workspace, size_t ws_bytes,
                moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  const Layout Y = layout(cfg);
  // INT8 mode reads wq alone
  const auto weight_ok = [&](const void* w) { return (Y.i8 && !w) || aligned16(w); };
  if (!aligned4(offsets) || !aligned4(tk_row) || !aligned4(topk_w) || !weight_ok(w1) ||
      !weight_ok(w2) || !aligned16(y) || !aligned16(saved) || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ring(Y, ring, ring_bytes, slot))) return st;
  if ((st = check_wq(Y, wq, wq_bytes))) return st;
  if (saved_bytes < Y.saved_total || ws_bytes < Y.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device())) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool pers = cfg->flags & MOE_FLAG_PERSISTENT;
  const int Tk = cfg->T * cfg->k, d = cfg->d, I = cfg->I, E = cfg->E;
  const uint8_t* slot_base = at<uint8_t>(ring, (size_t)slot * Y.slot);
  int2* sched = at<int2>(workspace, Y.sched);
  uint16_t* H = at<uint16_t>(saved, Y.H);
  uint16_t* A = at<uint16_t>(saved, Y.A);
  uint16_t* O = at<uint16_t>(workspace, Y.O);
  Launches L;
  if (Y.f8) {
    // the products find their row tiles from the offsets: no schedule table
    uint8_t* q = at<uint8_t>(workspace, Y.f8q);
    float* qs = at<float>(workspace, Y.f8s);
    L(launch_fp8_quant_rows(reinterpret_cast<const uint16_t*>(slot_base), Tk, d, q, qs, s));
    if (!L.err)
      L(launch_fp8_gemm({offsets, q, qs, at<uint8_t>(wq, Y.w1f), at<float>(wq, Y.w1fs), H, Tk, E,
                         2 * I, d},
                        s));
    if (!L.err) L(launch_fp8_swiglu(H, offsets + E, Tk, I, A, q, qs, s));
    if (!L.err)
      L(launch_fp8_gemm({offsets, q, qs, at<uint8_t>(wq, Y.w2f), at<float>(wq, Y.w2fs), O, Tk, E,
                         d, I},
                        s));
    if (!L.err)
      L(launch_combine(O, tk_row, topk_w, cfg->T, cfg->k, d, static_cast<uint16_t*>(y), s));
    return L.status();
  }
  if (Y.i8) {
    uint8_t* q = at<uint8_t>(workspace, Y.i8q);
    float* qs = at<float>(workspace, Y.i8s);
    L(launch_i8_quant_rows(reinterpret_cast<const uint16_t*>(slot_base), Tk, d, q, qs, s));
    if (!L.err)
      L(launch_i8_gemm({offsets, q, qs, at<uint8_t>(wq, Y.w1f), at<float>(wq, Y.w1fs), A, Tk, E,
                        2 * I, d, MOE_ACT_SILU},
                       true, s));
    if (!L.err) L(launch_i8_quant_rows(A, Tk, I, q, qs, s));
    if (!L.err)
      L(launch_i8_gemm({offsets, q, qs, at<uint8_t>(wq, Y.w2f), at<float>(wq, Y.w2fs), O, Tk, E, d,
                        I, 0},
                       false, s));
    if (!L.err)
      L(launch_combine(O, tk_row, topk_w, cfg->T, cfg->k, d, static_cast<uint16_t*>(y), s));
    return L.status();
  }
  L(launch_sched_build(offsets, E, Tk, sched, s));
  if (Y.mx) {
    uint8_t* aq = at<uint8_t>(workspace, Y.aq);
    uint8_t* aqs = at<uint8_t>(workspace, Y.aqs);
    if (!L.err)
      L(launch_fwd_gateup_mx({slot_base, slot_base + Y.slot_sc, at<uint8_t>(wq, Y.w1f),
                              at<uint8_t>(wq, Y.w1fs), H, A, aq, aqs, offsets, sched, d, I, Tk, E,
                              Y.fb},
                             pers, s));
    if (!L.err)
      L(launch_fwd_down_mx({aq, aqs, at<uint8_t>(wq, Y.w2f), at<uint8_t>(wq, Y.w2fs), O, offsets,
                            sched, d, I, Tk, E, Y.fb},
                           pers, s));
  } else {
    const uint16_t* xp = reinterpret_cast<const uint16_t*>(slot_base);
    if (!L.err)
      L(launch_fwd_gateup({xp, static_cast<const uint16_t*>(w1), H, A, offsets, sched, d, I, Tk, E},
                          pers, s));
    if (!L.err)
      L(launch_fwd_down({A, static_cast<const uint16_t*>(w2), O, offsets, sched, d, I, Tk, E}, pers,
                        s));
  }
  if (!L.err)
    L(launch_combine(O, tk_row, topk_w, cfg->T, cfg->k, d, static_cast<uint16_t*>(y), s));
  return L.status();
}

int moe_forward_fused(const moe_cfg* cfg, const void* x, const void* w_router, float* logits,
                      int32_t* topk_idx, float* topk_w, void* ring, size_t ring_bytes,
                      int32_t slot, int32_t* counts, int32_t* offsets, int32_t* row_src,
                      int32_t* tk_row, const void* w1, const void* w2, void* y, void* saved,
                      size_t saved_bytes, void* workspace, size_t ws_bytes, moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  if (cfg->precision != MOE_PREC_BF16) return MOE_ERR_UNSUPPORTED;
  const Layout Y = layout(cfg);
  if (!aligned16(x) || !aligned16(w_router) || !aligned4(logits) || !aligned4(topk_idx) ||
      !aligned4(topk_w) || !aligned4(counts) || !aligned4(offsets) || !aligned4(row_src) ||
      !aligned4(tk_row) || !aligned16(w1) || !aligned16(w2) || !aligned16(y) ||
      !aligned16(saved) || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ring(Y, ring, ring_bytes, slot))) return st;
  if (saved_bytes < Y.saved_total || ws_bytes < Y.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device())) return st;
  const int Tk = cfg->T * cfg->k;
  FusedFwdParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.wr = static_cast<const uint16_t*>(w_router);
  p.w32 = at<float>(workspace, Y.wr32);
  p.logits = logits;
  p.topk_idx = topk_idx;
  p.topk_w = topk_w;
  p.blk_cnt = at<int32_t>(workspace, Y.blk_cnt);
  p.rank = at<int32_t>(workspace, Y.rank);
  p.blk_flag = at<int32_t>(workspace, Y.blk_flag);
  p.counts = counts;
  p.offsets = offsets;
  p.status = at<int32_t>(workspace, Y.status);
  p.row_src = row_src;
  p.tk_row = tk_row;
  p.xp = at<uint16_t>(ring, (size_t)slot * Y.slot);
  p.sched = at<int2>(workspace, Y.sched);  // the 128-row block table opens the region
  p.w1 = static_cast<const uint16_t*>(w1);
  p.w2 = static_cast<const uint16_t*>(w2);
  p.H = at<uint16_t>(saved, Y.H);
  p.A = at<uint16_t>(saved, Y.A);
  p.O = at<uint16_t>(workspace, Y.O);
  p.y = static_cast<uint16_t*>(y);
  p.T = cfg->T;
  p.d = cfg->d;
  p.E = cfg->E;
  p.k = cfg->k;
  p.I = cfg->I;
  p.nb = Y.nb;
  // tokens per placement block, as moe_permute's launch chooses them
  int tpb = 1024 / (cfg->d / 8);
  if (tpb < 1) tpb = 1;
  if (tpb > 256 / cfg->k) tpb = 256 / cfg->k;
  p.tpb = tpb;
  (void)Tk;
  Launches L;
  L(launch_fused_forward(p, static_cast<hipStream_t>(stream)));
  return L.status();
}

int moe_backward(const moe_cfg* cfg, const void* ring, size_t ring_bytes, int32_t slot,
                 const int32_t* offsets, const int32_t* row_src, const int32_t* tk_row,
                 const int32_t* topk_idx, const float* topk_w, const void* w_router,
                 const void* w1, const void* w2, const void* wq, size_t wq_bytes,
                 const void* saved, size_t saved_bytes, const void* dy, void* dx, void* dw1,
                 void* dw2, float* dwr, float* d_topk_w, int32_t accumulate, void* workspace,
                 size_t ws_bytes, moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  if (cfg->precision == MOE_PREC_INT8) return MOE_ERR_UNSUPPORTED;
  const Layout Y = layout(cfg);
  const bool routed = w_router != nullptr;
  if (!aligned4(offsets) || !aligned4(row_src) || !aligned4(tk_row) || !aligned4(topk_idx) ||
      !aligned4(topk_w) || !aligned16(w1) || !aligned16(w2) || !aligned16(saved) ||
      !aligned16(dy) || !aligned16(dx) || !aligned16(dw1) || !aligned16(dw2) ||
      !aligned4(d_topk_w) || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  if (routed && (!aligned16(w_router) || !aligned16(dwr))) return MOE_ERR_INVALID_ARG;
  if ((st = check_ring(Y, ring, ring_bytes, slot))) return st;
  if ((st = check_wq(Y, wq, wq_bytes))) return st;
  if (saved_bytes < Y.saved_total || ws_bytes < Y.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device())) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool pers = cfg->flags & MOE_FLAG_PERSISTENT;
  const int bdw = (cfg->flags & MOE_FLAG_BF16_DW) ? 1 : 0;  // dW stored as bf16
  const int Tk = cfg->T * cfg->k, d = cfg->d, I = cfg->I, E = cfg->E, k = cfg->k;
  const uint8_t* slot_base = at<uint8_t>(ring, (size_t)slot * Y.slot);
  const uint16_t* xp = Y.mx ? nullptr : reinterpret_cast<const uint16_t*>(slot_base);
  const uint8_t* xp8 = Y.mx ? slot_base : nullptr;
  const uint8_t* xps = Y.mx ? slot_base + Y.slot_sc : nullptr;
  const uint16_t* H = at<uint16_t>(saved, Y.H);
  const uint16_t* A = at<uint16_t>(saved, Y.A);
  int2* sched = at<int2>(workspace, Y.sched);
  uint16_t* dH = at<uint16_t>(workspace, Y.dH);
  uint16_t* dXp = at<uint16_t>(workspace, Y.dXp);
  float* dwpart = at<float>(workspace, Y.dwpart);
  float* dl_pos = at<float>(workspace, Y.dl_pos);
  uint16_t* dyw = at<uint16_t>(workspace, Y.dyw);
  int32_t* wg_count = at<int32_t>(workspace, Y.wg_count);
  const uint16_t* dyp = static_cast<const uint16_t*>(dy);
  const uint16_t* w1p = static_cast<const uint16_t*>(w1);
  const uint16_t* w2p = static_cast<const uint16_t*>(w2);
  Launches L;
  if (!Y.f8) L(launch_sched_build(offsets, E, Tk, sched, s));
  if (Y.f8) {
    uint8_t* q = at<uint8_t>(workspace, Y.f8q);
    float* qs = at<float>(workspace, Y.f8s);
    uint16_t* dAp = at<uint16_t>(workspace, Y.dAp);
    L(launch_scale_gather(dyp, tk_row, topk_w, cfg->T, k, d, dyw, s));
    if (!L.err) L(launch_fp8_quant_gather(dyp, row_src, k, offsets + E, Tk, d, q, qs, s));
    if (!L.err)
      L(launch_fp8_gemm({offsets, q, qs, at<uint8_t>(wq, Y.w2b), at<float>(wq, Y.w2bs), dAp, Tk, E,
                         I, d},
                        s));
    if (!L.err)
      L(launch_fp8_swiglu_bwd({dAp, H, A, row_src, topk_w, offsets + E, Tk, I, dH, q, qs, dwpart},
                              s));
    if (!L.err)
      L(launch_dw_router(dwpart, Y.nIt, tk_row, topk_w, cfg->T, k, d_topk_w, dl_pos, routed, s));
    if (!L.err)
      L(launch_wgrad({dyw, A, nullptr, nullptr, dw2, offsets, at<int4>(workspace, Y.wg_table2),
                      wg_count + 1, E, d, I, accumulate, bdw, false, "bwd_down_wgrad",
                      "wgrad_sched_down"},
                     s));
    if (!L.err)
      L(launch_fp8_gemm({offsets, q, qs, at<uint8_t>(wq, Y.w1b), at<float>(wq, Y.w1bs), dXp, Tk, E,
                         d, 2 * I},
                        s));
    if (!L.err)
      L(launch_wgrad({dH, xp, nullptr, nullptr, dw1, offsets, at<int4>(workspace, Y.wg_table1),
                      wg_count, E, 2 * I, d, accumulate, bdw, true, "bwd_gate_wgrad",
                      "wgrad_sched_gate"},
                     s));
  } else if (Y.mx) {
    uint8_t* dyq = at<uint8_t>(workspace, Y.dyq);
    uint8_t* dys = at<uint8_t>(workspace, Y.dys);
    uint8_t* dhq = at<uint8_t>(workspace, Y.dhq);
    uint8_t* dhs = at<uint8_t>(workspace, Y.dhs);
    if (!L.err) L(launch_quant_rows(dyp, cfg->T, d, dyq, dys, Y.fb, "quant_dy", s));
    if (!L.err) L(launch_scale_gather(dyp, tk_row, topk_w, cfg->T, k, d, dyw, s));
    if (!L.err)
      L(launch_bwd_down_dgrad_mx({dyq, dys, row_src, topk_w, at<uint8_t>(wq, Y.w2b),
                                  at<uint8_t>(wq, Y.w2bs), H, A, dH, dwpart, dhq, dhs, offsets,
                                  sched, d, I, k, Tk, E, Y.fb},
                                 pers, s));
    if (!L.err)
      L(launch_dw_router(dwpart, Y.nIt, tk_row, topk_w, cfg->T, k, d_topk_w, dl_pos, routed, s));
    if (cfg->flags & MOE_FLAG_MXFP8_WGRAD) {
      // both weight gradients in MXFP8, their operands quantised along each expert's positions
      int32_t* poff = at<int32_t>(workspace, Y.poff);
      uint8_t* lq = at<uint8_t>(workspace, Y.lq);
      uint8_t* lqs = at<uint8_t>(workspace, Y.lqs);
      uint8_t* rq = at<uint8_t>(workspace, Y.rq);
      uint8_t* rqs = at<uint8_t>(workspace, Y.rqs);
      if (!L.err) L(launch_seg_offsets(offsets, E, poff, s));
      SegOperand wdy, sa, sdh, sxp;
      wdy.src = dyp;  // w * dY, formed in fp32 and quantised from that
      wdy.row_src = row_src;
      wdy.topk_w = topk_w;
      wdy.k = k;
      sa.src = A;
      sdh.src = dH;
      sxp.src8 = xp8;
      sxp.src8s = xps;
      if (!L.err)
        L(launch_quant_seg(wdy, offsets, poff, E, d, Y.P, lq, lqs, "bwd_down_wgrad_qL", s));
      if (!L.err)
        L(launch_quant_seg(sa, offsets, poff, E, I, Y.P, rq, rqs, "bwd_down_wgrad_qR", s));
      if (!L.err)
        L(launch_mx_wgrad({lq, lqs, rq, rqs, dw2, poff, E, d, I, Y.P, accumulate, bdw,
                           "bwd_down_wgrad"},
                          pers, s));
      if (!L.err)
        L(launch_quant_seg(sdh, offsets, poff, E, 2 * I, Y.P, lq, lqs, "bwd_gate_wgrad_qL", s));
      if (!L.err)
        L(launch_quant_seg(sxp, offsets, poff, E, d, Y.P, rq, rqs, "bwd_gate_wgrad_qR", s));
      if (!L.err)
        L(launch_mx_wgrad({lq, lqs, rq, rqs, dw1, poff, E, 2 * I, d, Y.P, accumulate, bdw,
                           "bwd_gate_wgrad"},
                          pers, s));
    } else {
      if (!L.err)
        L(launch_wgrad({dyw, A, nullptr, nullptr, dw2, offsets, at<int4>(workspace, Y.wg_table2),
                        wg_count + 1, E, d, I, accumulate, bdw, false, "bwd_down_wgrad",
                        "wgrad_sched_down"},
                       s));
      // the gate wgrad goes first: until the gate dgrad writes dXp, that buffer holds the bf16
      // image of the big experts' MX Xp rows for the big-expert wgrad kernel
      if (!L.err)
        L(launch_wgrad({dH, nullptr, xp8, xps, dw1, offsets, at<int4>(workspace, Y.wg_table1),
                        wg_count, E, 2 * I, d, accumulate, bdw, true, "bwd_gate_wgrad",
                        "wgrad_sched_gate", dXp, Y.fb},
                       s));
    }
    if (!L.err)
      L(launch_bwd_gate_dgrad_mx({dhq, dhs, at<uint8_t>(wq, Y.w1b), at<uint8_t>(wq, Y.w1bs), dXp,
                                  offsets, sched, d, I, Tk, E, Y.fb},
                                 pers, s));
  } else {
    if (!L.err) L(launch_scale_gather(dyp, tk_row, topk_w, cfg->T, k, d, dyw, s));
    if (!L.err)
      L(launch_bwd_down_dgrad({dyp, row_src, topk_w, w2p, H, A, dH, dwpart, offsets, sched, d, I,
                               k, Tk, E},
                              pers, s));
    if (!L.err)
      L(launch_dw_router(dwpart, Y.nIt, tk_row, topk_w, cfg->T, k, d_topk_w, dl_pos, routed, s));
    if (!L.err)
      L(launch_wgrad({dyw, A, nullptr, nullptr, dw2, offsets, at<int4>(workspace, Y.wg_table2),
                      wg_count + 1, E, d, I, accumulate, bdw, false, "bwd_down_wgrad",
                      "wgrad_sched_down"},
                     s));
    if (!L.err) L(launch_bwd_gate_dgrad({dH, w1p, dXp, offsets, sched, d, I, Tk, E}, pers, s));
    if (!L.err)
      L(launch_wgrad({dH, xp, nullptr, nullptr, dw1, offsets, at<int4>(workspace, Y.wg_table1),
                      wg_count, E, 2 * I, d, accumulate, bdw, true, "bwd_gate_wgrad",
                      "wgrad_sched_gate"},
                     s));
  }
  if (!L.err)
    L(launch_uncombine(dXp, tk_row, topk_idx, dl_pos,
                       routed ? static_cast<const uint16_t*>(w_router) : nullptr, cfg->T, k, d,
                       static_cast<uint16_t*>(dx), s));
  if (!L.err && routed) L(launch_dwr(dl_pos, xp, xp8, xps, Y.fb, offsets, E, d, dwr, accumulate, s));
  return L.status();
}

int moe_gate_select(const moe_cfg* cfg, const moe_gate* gate, const float* logits,
                    const float* bias, int32_t* topk_idx, float* topk_w, moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  if ((st = check_gate(cfg, gate))) return st;
  if (!aligned4(logits) || (bias && !aligned4(bias)) || !aligned4(topk_idx) || !aligned4(topk_w))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_device())) return st;
  Launches L;
  L(launch_gate_select(gate_params(gate), logits, bias, cfg->T, cfg->E, cfg->k, topk_idx, topk_w,
                       static_cast<hipStream_t>(stream)));
  return L.status();
}

int moe_route_gated(const moe_cfg* cfg, const moe_gate* gate, const void* x, const void* w_router,
                    const float* bias, float* logits, int32_t* topk_idx, float* topk_w,
                    void* workspace, size_t ws_bytes, moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  if ((st = check_gate(cfg, gate))) return st;
  if (!aligned16(x) || !aligned16(w_router) || (bias && !aligned4(bias)) || !aligned4(logits) ||
      !aligned4(topk_idx) || !aligned4(topk_w) || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  const Layout Y = layout(cfg);
  if (ws_bytes < Y.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device())) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Launches L;
  L(launch_router_logits(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w_router),
                         at<float>(workspace, Y.wr32), logits, cfg->T, cfg->d, cfg->E, s));
  if (!L.err)
    L(launch_gate_select(gate_params(gate), logits, bias, cfg->T, cfg->E, cfg->k, topk_idx, topk_w,
                         s));
  return L.status();
}

int moe_gate_backward(const moe_cfg* cfg, const moe_gate* gate, const float* logits,
                      const int32_t* topk_idx, const float* d_topk_w, float* dlogits,
                      int32_t accumulate, moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  if ((st = check_gate(cfg, gate))) return st;
  if (!aligned4(logits) || !aligned4(topk_idx) || !aligned4(d_topk_w) || !aligned4(dlogits))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_device())) return st;
  Launches L;
  L(launch_gate_backward(gate_params(gate), logits, topk_idx, d_topk_w, cfg->T, cfg->E, cfg->k,
                         dlogits, accumulate, static_cast<hipStream_t>(stream)));
  return L.status();
}

int moe_router_backward(const moe_cfg* cfg, const void* x, const void* w_router,
                        const float* dlogits, void* dx, float* dwr, int32_t acc_dx,
                        int32_t acc_dwr, moe_stream_t stream) {
  int st = check_mode(cfg);
  if (st) return st;
  if (!aligned16(x) || !aligned16(w_router) || !aligned4(dlogits) || (dx && !aligned16(dx)) ||
      (dwr && !aligned16(dwr)) || (!dx && !dwr) || dx == x)
    return MOE_ERR_INVALID_ARG;
  if ((st = check_device())) return st;
  RouterGradArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w_router),
                   dlogits, static_cast<uint16_t*>(dx), dwr, cfg->T, cfg->d, cfg->E, acc_dx,
                   acc_dwr};
  Launches L;
  L(launch_router_backward(a, static_cast<hipStream_t>(stream)));
  return L.status();
}

int moe_fp8_quantize_rows(const void* src, int32_t rows, int32_t cols, void* codes, float* scales,
                          moe_stream_t stream) {
  if (rows < 0 || cols < 128 || cols % 128 != 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;  // empty buffers have no address to check
  if (!aligned16(src) || !aligned16(codes) || !aligned4(scales)) return MOE_ERR_INVALID_ARG;
  // the grid: a workgroup for 32 rows x 512 columns, and fewer than 2^32 threads
  if ((rows + 31LL) / 32 * ((cols + 511LL) / 512) >= (1LL << 24)) return MOE_ERR_INVALID_ARG;
  if (const int st = check_device()) return st;
  Launches L;
  L(launch_fp8_quant_rows(static_cast<const uint16_t*>(src), rows, cols,
                          static_cast<uint8_t*>(codes), scales,
                          static_cast<hipStream_t>(stream)));
  return L.status();
}

int moe_fp8_quantize_weights(const void* src, int32_t E, int32_t N, int32_t K, void* codes,
                             float* scales, void* codes_t, float* scales_t, moe_stream_t stream) {
  if (const int st = check_fp8_shape(E, N, K)) return st;
  if (!aligned16(src) || !aligned16(codes) || !aligned4(scales) || !codes_t != !scales_t ||
      (codes_t && (!aligned16(codes_t) || !aligned4(scales_t))))
    return MOE_ERR_INVALID_ARG;
  if (const int st = check_device()) return st;
  Launches L;
  L(launch_fp8_quant_weights(static_cast<const uint16_t*>(src), E, N, K,
                             static_cast<uint8_t*>(codes), scales, static_cast<uint8_t*>(codes_t),
                             scales_t, static_cast<hipStream_t>(stream)));
  return L.status();
}

int moe_fp8_gemm(const int32_t* offsets, int32_t M, int32_t E, int32_t N, int32_t K, const void* a,
                 const float* a_scales, const void* b, const float* b_scales, void* out,
                 moe_stream_t stream) {
  if (const int st = check_fp8_shape(E, N, K)) return st;
  if (M < 0 || !aligned4(offsets) || !aligned16(b) || !aligned4(b_scales))
    return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;  // empty buffers have no address to check
  if (!aligned16(a) || !aligned4(a_scales) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  if ((M / 16LL + E) * (N / 128) >= (1LL << 31)) return MOE_ERR_INVALID_ARG;  // the grid
  if (const int st = check_device()) return st;
  Fp8GemmArgs g{offsets, static_cast<const uint8_t*>(a), a_scales,
                static_cast<const uint8_t*>(b), b_scales, static_cast<uint16_t*>(out), M, E, N, K};
  Launches L;
  L(launch_fp8_gemm(g, static_cast<hipStream_t>(stream)));
  return L.status();
}

int moe_i8_quantize_rows(const void* src, int32_t rows, int32_t cols, void* codes, float* scales,
                         moe_stream_t stream) {
  if (rows < 0 || rows >= (1 << 24) || cols < 128 || cols % 128 != 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;  // empty buffers have no address to check
  if (!aligned16(src) || !aligned16(codes) || !aligned4(scales)) return MOE_ERR_INVALID_ARG;
  if (const int st = check_device()) return st;
  Launches L;
  L(launch_i8_quant_rows(static_cast<const uint16_t*>(src), rows, cols,
                         static_cast<uint8_t*>(codes), scales, static_cast<hipStream_t>(stream)));
  return L.status();
}

int moe_i8_gemm(const int32_t* offsets, int32_t M, int32_t E, int32_t N, int32_t K, const void* a,
                const float* a_scales, const void* b, const float* b_scales, void* out,
                moe_stream_t stream) {
  return i8_gemm(offsets, M, E, N, K, 0, false, a, a_scales, b, b_scales, out, stream);
}

int moe_i8_gemm_gated(const int32_t* offsets, int32_t M, int32_t E, int32_t I, int32_t K,
                      int32_t act, const void* a, const float* a_scales, const void* b,
                      const float* b_scales, void* out, moe_stream_t stream) {
  if (I < 128 || I % 128 != 0 || I >= (1 << 30) || !act_ok(act)) return MOE_ERR_INVALID_ARG;
  return i8_gemm(offsets, M, E, 2 * I, K, act, true, a, a_scales, b, b_scales, out, stream);
}

int moe_ffn_query(const moe_ffn* ffn, moe_ffn_sizes* out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  if (const int st = check_ffn(ffn)) return st;
  out->workspace = ffn_layout(ffn).total;
  return MOE_OK;
}

int moe_ffn_forward(const moe_ffn* ffn, const void* x, const void* w1, const void* w2, void* H,
                    void* A, void* y, int32_t acc_y, void* workspace, size_t ws_bytes,
                    moe_stream_t stream) {
  if (const int st = check_ffn(ffn)) return st;
  if (!aligned16(x) || !aligned16(w1) || !aligned16(w2) || (H && !aligned16(H)) ||
      !aligned16(A) || !aligned16(y) || y == x || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  const FfnLayout Y = ffn_layout(ffn);
  if (ws_bytes < Y.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (const int st = check_device()) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  FfnArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.w1 = static_cast<const uint16_t*>(w1);
  a.w2 = static_cast<const uint16_t*>(w2);
  a.H = static_cast<uint16_t*>(H);
  a.A = static_cast<uint16_t*>(A);
  a.y = static_cast<uint16_t*>(y);
  a.T = ffn->T;
  a.d = ffn->d;
  a.I = ffn->I;
  a.act = ffn->act;
  a.part = at<float>(workspace, Y.part);
  a.acc_y = acc_y != 0;
  Launches L;
  L(launch_ffn_gate_up(a, s));
  if (!L.err) L(launch_ffn_down(a, s));
  return L.status();
}

int moe_ffn_backward(const moe_ffn* ffn, const void* x, const void* w1, const void* w2,
                     const void* H, const void* A, const void* dy, void* dx, void* dw1, void* dw2,
                     int32_t acc_dx, int32_t acc_dw, void* workspace, size_t ws_bytes,
                     moe_stream_t stream) {
  if (const int st = check_ffn(ffn)) return st;
  if (!aligned16(x) || !aligned16(w1) || !aligned16(w2) || !aligned16(H) || !aligned16(A) ||
      !aligned16(dy) || !aligned16(dx) || !aligned16(dw1) || !aligned16(dw2) || dx == x ||
      dx == dy || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  const FfnLayout Y = ffn_layout(ffn);
  if (ws_bytes < Y.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (const int st = check_device()) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int bdw = ffn->flags & MOE_FLAG_BF16_DW ? 1 : 0, acc = acc_dw != 0;
  FfnArgs a{};
  a.w1 = static_cast<const uint16_t*>(w1);
  a.w2 = static_cast<const uint16_t*>(w2);
  a.H = const_cast<uint16_t*>(static_cast<const uint16_t*>(H));
  a.dy = static_cast<const uint16_t*>(dy);
  a.dH = at<uint16_t>(workspace, Y.dH);
  a.part = at<float>(workspace, Y.part);
  a.dx = static_cast<uint16_t*>(dx);
  a.T = ffn->T;
  a.d = ffn->d;
  a.I = ffn->I;
  a.act = ffn->act;
  a.acc_dx = acc_dx != 0;
  Launches L;
  float* part = at<float>(workspace, Y.part_dw);
  L(launch_ffn_dh_dw2(
      a, {a.dy, static_cast<const uint16_t*>(A), dw2, part, a.T, a.d, a.I, acc, bdw, 1}, s));
  if (!L.err)
    L(launch_ffn_dx_dw1(
        a, {a.dH, static_cast<const uint16_t*>(x), dw1, part, a.T, 2 * a.I, a.d, acc, bdw, 1}, s));
  return L.status();
}

const char* moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_RING_TOO_SMALL: return "ring buffer too small for the requested slot";
    case MOE_ERR_UNSUPPORTED: return "unsupported mode";
    case MOE_ERR_HIP: return "HIP runtime error while enqueuing";
    case MOE_ERR_WORKSPACE_TOO_SMALL: return "workspace or saved buffer too small";
    default: return "unknown status";
  }
}

}  // extern "C"
