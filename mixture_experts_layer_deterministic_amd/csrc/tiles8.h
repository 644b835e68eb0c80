// What the products that feed 128-byte K steps straight into LDS share (fp8.hip, int8.hip, ffn.hip):
// the experts' row tiles, the loads, and the places of the codes in LDS.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kCus = 256;   // MI355X; tiles that run at once
constexpr int kBigT = 256;  // rows and columns of the largest tiles
typedef __attribute__((ext_vector_type(4))) int i32x4;

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

// LDS tiles of 128-byte rows (one block of K), 16-byte chunk c of row r at c ^ (r & 7), so that
// fragment reads spread over the banks. A lane's operand of the 16 x 16 x 128 MFMA: chunks g and
// 4 + g of row l % 16 of a block of 16 rows, g = l / 16. Rows and columns take the same k in the
// same place, which is all a sum over the whole block needs. The two byte offsets are the same
// in every row block, so the blocks differ by constants.
struct FragAt {
  int lo, hi;
};
MOE_DEV FragAt frag_at(int lane) {
  const int r = lane % 16, g = lane / 16;
  return {r * 128 + ((g ^ (r & 7)) << 4), r * 128 + (((4 + g) ^ (r & 7)) << 4)};
}
MOE_DEV __amdgpu_buffer_rsrc_t buf_rsrc(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, 0x00020000);
}
// 16 bytes a lane straight into LDS, at lds + 16 lane: 8 rows of 128 bytes a wave.
template <int AUX = 0>
MOE_DEV void load_lds16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                           voff, soff, 0, AUX);
}
// The chunk a lane fetches into its place of those 8 rows.
MOE_DEV uint32_t lds_piece(int lane) { return 16u * ((lane % 8) ^ (lane / 8)); }

// Behind it no load goes out before those in front of it: what a counted wait relies on.
MOE_DEV void loads_in_order() { __builtin_amdgcn_sched_barrier(0x40f); }  // arithmetic may pass

constexpr int kVm4Lgkm0 = 0x0074;  // s_waitcnt vmcnt(4) lgkmcnt(0)
constexpr int kVm0Lgkm0 = 0x0070;  // s_waitcnt vmcnt(0) lgkmcnt(0)
constexpr int kLgkm0 = 0xc07f;     // lgkmcnt(0) alone

// The experts' row tiles counted out: all of them, and the one with a given number.
template <class G>  // arguments of a grouped product: offsets, M, E
MOE_DEV int big_tiles_of(const G& a, int e) {
  if (e >= a.E) return 0;
  const int lo = min(max(a.offsets[e], 0), a.M), hi = min(max(a.offsets[e + 1], 0), a.M);
  return hi > lo ? (hi - lo + kBigT - 1) / kBigT : 0;
}
MOE_DEV int wave_scan(int v) {
  const int lane = threadIdx.x % kWave;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int u = __shfl_up(v, o);
    v += lane >= o ? u : 0;
  }
  return v;
}
template <class G>
MOE_DEV int big_count(const G& a) {
  int n = 0;
  for (int e0 = 0; e0 < a.E; e0 += kWave)
    n += __builtin_amdgcn_readlane(wave_scan(big_tiles_of(a, e0 + threadIdx.x % kWave)), 63);
  return n;
}
template <class G>
MOE_DEV RowTile big_rows(const G& a, int mt) {
  RowTile t{0, 0, 0};
  for (int e0 = 0; e0 < a.E; e0 += kWave) {
    const int inc = wave_scan(big_tiles_of(a, e0 + threadIdx.x % kWave));
    const int all = __builtin_amdgcn_readlane(inc, 63);
    if (mt < all) {
      const int n = __popcll(__ballot(inc <= mt));  // experts before the tile's
      t.e = e0 + n;
      const int i = mt - (n ? __builtin_amdgcn_readlane(inc, n - 1) : 0);
      const int lo = min(max(a.offsets[t.e], 0), a.M), hi = min(max(a.offsets[t.e + 1], 0), a.M);
      t.row0 = lo + i * kBigT;
      t.rows = min(hi - t.row0, kBigT);
      return t;
    }
    mt -= all;
  }
  return t;
}
// Tile number -> (row tile, column tile): four row tiles take each column tile in turn, so that
// the tiles an XCD runs at once (32) share few panels of either operand in its L2.
MOE_DEV int2 big_order(int lt, int nm, int nN) {
  const int first = lt / (4 * nN) * 4, gm = min(4, nm - first), r = lt - first * nN;
  return make_int2(first + r % gm, r / gm);
}

}  // namespace
}  // namespace moe
