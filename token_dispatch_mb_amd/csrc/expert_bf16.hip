// expert_bf16.hip — the experts' feed-forward products from bf16 rows and
// weights, and their gradients (mb_expert_bf16, mb_expert_bf16_dgrad,
// mb_expert_bf16_wgrad).
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

// 128 or 256 rows to a tile, from the rows expected in a slot.
template <int kMode, bool kBF16>
void launch_tiles(const TileArgs& p, int64_t rows, hipStream_t st) {
  const int64_t slots = (int64_t)p.P * p.NS;
  const int64_t columns = (p.n + kTileN - 1) / kTileN;
  const dim3 grid(kCus), block(kExpertThreads);
  if constexpr (kMode == kTileProduct || kMode == kTileGated) {
    if (rows < slots * 2) {
      hipLaunchKernelGGL((k_bf16_few<kMode, kBF16, 4, 4>), dim3(kFewGroups), block, 0, st, p);
      return;
    }
  }
  if (rows >= slots * 160 && (rows / 256 + slots) * columns > 2 * kCus)
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
  // 256 rows to a tile where they occupy the CUs
  const int64_t tiles = (int64_t)p.E * ((p.k + 255) / 256) * ((p.n + kTileN - 1) / kTileN);
#define MB_W(BF16, JT)                                                                       \
  do {                                                                                       \
    if (add)                                                                                 \
      hipLaunchKernelGGL((k_bf16_tile<kTileWeightAdd, BF16, JT>), grid, block, 0, st, p);    \
    else                                                                                     \
      hipLaunchKernelGGL((k_bf16_tile<kTileWeightGrad, BF16, JT>), grid, block, 0, st, p);   \
  } while (0)
  const dim3 grid(kCus), block(kExpertThreads);
  if (tiles >= kCus) {
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
