// expert_bf16.hip — the experts' feed-forward products from bf16 rows and
// weights, and their gradients (mb_expert_bf16, mb_expert_bf16_dgrad,
// mb_expert_bf16_wgrad).
//
//   y = a w[e]^T, or silu(g) u of its two halves; da = dy w[e], or times the
//   activation's derivatives; dw[e] = sum of dy^T a over e's rows.
//
// The activation and its gradient are in the products' stores, so that gate,
// up and their gradients pass memory once. A weight's gradient walks all slots
// that hold its expert in one sum: replicas need no second pass, and the order
// of the sum is the plan's.
#include "bf16_tile.h"

namespace mb {
namespace {

constexpr int kFewGroups = 2048;

TileArgs plan_args(const mb_dims& d, const Geometry& g, const mb_plan_bufs& o) {
  TileArgs p = {};
  p.cu = o.cu_seqlens;
  p.rep = o.rep_expert;
  p.status = o.status;
  p.P = d.n_ranks, p.E = d.n_experts, p.Eh = g.Eh, p.NS = g.NS, p.R = d.slots_per_rank;
  p.cap = d.cap;
  return p;
}

// Whether 256 rows to a tile take less time than 128: in rounds over the CUs,
// of which one of 256 rows takes kLongTile / 8 times as long.
bool long_tiles(int64_t tiles256, int64_t tiles128) {
  return (tiles256 + kCus - 1) / kCus * kLongTile <= (tiles128 + kCus - 1) / kCus * 8;
}

// From the rows expected in a slot, and 32 more, half of the 64 that tiles leave
// out of a slot's last one at a time.
//
// Few rows, straight from memory: up to eight in a slot, or where the columns
// of tiles, times the 16-row blocks that would each pass the weights, are fewer
// than half the CUs, since tiles leave the rest idle. us, against tiles:
//   7168 -> 2 x 3200 and back (25 and 28 columns): 1 slot, 9 rows 25 + 15, 79 +
//     41; 32 rows 43 + 27, 79 + 42; 64 rows 79 + 44, 80 + 42. 4 slots, 9 rows 94
//     + 37, 109 + 47; 24 rows 147 + 76, 110 + 47. 8 slots, 8 rows 164 + 83, 130
//     + 67 (the rule misses this one); 9 rows 166 + 86, 130 + 67.
//   4096 -> 2 x 2048 and back (16 and 16): 1 slot, 64 rows 27 + 19, 45 + 24; 128
//     rows 48 + 33, 51 + 28. 8 slots, 24 rows 91 + 56, 64 + 33. 64 slots, 4 rows
//     387 + 202, 547 + 230; 8 rows 410 + 230, 551 + 231; 16 rows 467 + 279, 552 +
//     232.
//   8192 -> 2048 (8): 1 slot, 128 rows 61, 83; 256 rows 118, 86. 7168 -> 256 (1): 1
//     slot, 1024 rows 55, 75; 1700 rows 92, 76 (missed).
// The rows' gradients have tiles only, which few slots leave idle too: 7168 x
// 3200, 1 slot 66 and 77 us at 4 as at 64 rows, 8 slots 106 and 129.
// 128 and 256 rows to a tile, 64 slots: 4096 rows 706 and 715 us, 8192 rows
// 795 and 768, 32768 rows 1830 and 1617; one slot, 7168 x 4096 and back: 1024
// rows 180 and 277, 2048 rows 326 and 290, 4096 rows 627 and 562.
template <int kMode, bool kBF16>
void launch_tiles(const TileArgs& p, int64_t rows, hipStream_t st) {
  const int64_t slots = (int64_t)p.P * p.NS;
  const int64_t across = kMode == kTileGated ? kTileN / 2 : kTileN;
  const int64_t columns = (p.n + across - 1) / across;
  const dim3 grid(kCus), block(kExpertThreads);
  if constexpr (kMode == kTileProduct || kMode == kTileGated) {
    const int64_t blocks = (rows + slots * 16 - 1) / (slots * 16) * slots;
    if (rows <= slots * 8 || blocks * columns < kCus / 2) {
      hipLaunchKernelGGL((k_bf16_few<kMode, kBF16, 4, 4>), dim3(kFewGroups), block, 0, st, p);
      return;
    }
  }
  const int64_t all = rows + slots / 2 * 64;
  auto tiles = [&](int64_t tall) { return (all + tall - 1) / tall * columns; };
  if (rows >= slots * 128 && long_tiles(tiles(256), tiles(128)))
    hipLaunchKernelGGL((k_bf16_tile<kMode, kBF16, 4>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((k_bf16_tile<kMode, kBF16, 2>), grid, block, 0, st, p);
}

}  // namespace

hipError_t launch_expert_bf16(const mb_dims& d, const Geometry& g, const mb_plan_bufs& o,
                              bool gated, int32_t n_out, int32_t k_in, const uint16_t* a,
                              const uint16_t* w, void* y, uint16_t* pre, hipStream_t st) {
  if (d.n_tokens == 0) return hipSuccess;
  TileArgs p = plan_args(d, g, o);
  p.a = a, p.w = w, p.y = y, p.pre = pre, p.n = n_out, p.k = k_in;
  const int64_t rows = (int64_t)d.n_tokens * d.top_k;
  if (gated)
    launch_tiles<kTileGated, true>(p, rows, st);
  else if (d.dtype_out == MB_BF16)
    launch_tiles<kTileProduct, true>(p, rows, st);
  else
    launch_tiles<kTileProduct, false>(p, rows, st);
  return hipGetLastError();
}

hipError_t launch_expert_bf16_dgrad(const mb_dims& d, const Geometry& g, const mb_plan_bufs& o,
                                    bool gated, int32_t n_out, int32_t k_in, const uint16_t* dy,
                                    const uint16_t* w, const uint16_t* pre, void* da,
                                    hipStream_t st) {
  if (d.n_tokens == 0) return hipSuccess;
  TileArgs p = plan_args(d, g, o);
  p.a = dy, p.w = w, p.y = da, p.pre = const_cast<uint16_t*>(pre), p.n = k_in, p.k = n_out;
  const int64_t rows = (int64_t)d.n_tokens * d.top_k;
  if (gated)
    launch_tiles<kTileGateGrad, true>(p, rows, st);
  else if (d.dtype_out == MB_BF16)
    launch_tiles<kTileRowGrad, true>(p, rows, st);
  else
    launch_tiles<kTileRowGrad, false>(p, rows, st);
  return hipGetLastError();
}

hipError_t launch_expert_bf16_wgrad(const mb_dims& d, const Geometry& g, const mb_plan_bufs& o,
                                    int32_t n_out, int32_t k_in, bool add, bool bf16,
                                    const uint16_t* dy, const uint16_t* a, void* dw,
                                    hipStream_t st) {
  TileArgs p = plan_args(d, g, o);
  p.a = dy, p.w = a, p.y = dw, p.n = k_in, p.k = n_out;
  if (d.n_tokens == 0) p.cap = 0;  // no rows, though the plan be of another call
  // (one expert, 2048 rows, both gradients: 4096 x 4096 151 us with 128 rows to
  // a tile, 137 with 256; 4096 x 2048, half the tiles, 106 and 171)
  auto tiles = [&](int64_t tall) {
    return (int64_t)p.E * ((p.k + tall - 1) / tall) * ((p.n + kTileN - 1) / kTileN);
  };
#define MB_W(BF16, JT)                                                                       \
  do {                                                                                       \
    if (add)                                                                                 \
      hipLaunchKernelGGL((k_bf16_tile<kTileWeightAdd, BF16, JT>), grid, block, 0, st, p);    \
    else                                                                                     \
      hipLaunchKernelGGL((k_bf16_tile<kTileWeightGrad, BF16, JT>), grid, block, 0, st, p);   \
  } while (0)
  const dim3 grid(kCus), block(kExpertThreads);
  if (long_tiles(tiles(256), tiles(128))) {
    if (bf16) MB_W(true, 4);
    else MB_W(false, 4);
  } else {
    if (bf16) MB_W(true, 2);
    else MB_W(false, 2);
  }
#undef MB_W
  return hipGetLastError();
}

}  // namespace mb
