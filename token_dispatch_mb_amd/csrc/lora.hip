// lora.hip — a projection with the low-rank adapters of many requests beside
// it (mb_project_lora).
//
//   y[t] = x[t] w^T + v[t] b_a^T,  v[t] = scale_a x[t] a_a^T,  a = adapter[t]
//
// k_lora_down makes v, in binary32; the product then goes on over the ranks
// of the adapters among a tile's rows, so that w and y are passed once.
#include <algorithm>

#include "bf16_tile.h"

namespace mb {
namespace {

constexpr int kFewGroups = 2048;
constexpr int kDownStep = 128;

struct DownArgs {
  const uint16_t* x;
  const uint16_t* a;  // [L][rank][k]
  const float* scale;
  const int32_t* adapter;
  float* v;  // [parts][rows][rank]
  int rows, k, rank, L, parts;
};

// v of 16 MT rows and 16 RT ranks, of one of their adapters or of one after
// the other: workgroup (x, y, z) takes the row block x, adapters y, y +
// gridDim.y, ... in the order of their numbers, and part z of the reduction.
// Its four waves take 128 elements by turns and add up in LDS. Rows without an
// adapter are not written (nothing reads them). MT = 4 passes a third as much
// of the adapters through the caches as MT = 1.
template <int RT, int MT>
__global__ __launch_bounds__(kExpertThreads) void k_lora_down(DownArgs p) {
  constexpr int U = kDownStep / 32;
  __shared__ f32x4 sums[4][RT * MT][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  int row[MT], id[MT];
  const uint16_t* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    row[i] = (blockIdx.x * MT + i) * 16 + r;
    const int at = min(row[i], p.rows - 1);
    id[i] = p.adapter[at];
    if ((unsigned)id[i] >= (unsigned)p.L || row[i] >= p.rows) id[i] = INT32_MAX;
    x[i] = p.x + (int64_t)at * p.k + g * 8;
  }
  // part z: whole turns of four waves
  const int turns = (p.k + 4 * kDownStep - 1) / (4 * kDownStep);
  const int each = (turns + p.parts - 1) / p.parts;
  const int k0 = min((int)blockIdx.z * each * 4 * kDownStep, p.k);
  const int k1 = min(k0 + each * 4 * kDownStep, p.k);
  int ad = -1;
  for (int j = 0;; ++j) {
    int least = INT32_MAX;
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (id[i] > ad) least = min(least, id[i]);
    ad = wave_min_i32(least);
    if (ad == INT32_MAX) break;
    if (j % gridDim.y != blockIdx.y) continue;
    const float scale = p.scale[ad];
    for (int q = 0; q < p.rank; q += 16 * RT) {
      const uint16_t* a[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
        a[i] = p.a + ((int64_t)ad * p.rank + min(q + i * 16 + r, p.rank - 1)) * p.k + g * 8;
      f32x4 acc[RT][MT] = {};
      int k = k0 + wave * kDownStep;
      // the next turn's operands are under way while this one's are multiplied
      i32x4 xv[2][MT][U], av[2][RT][U];
      auto fetch = [&](int to, int at) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int u = 0; u < U; ++u) xv[to][m][u] = load16(x[m] + at + u * 32);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int u = 0; u < U; ++u) av[to][i][u] = load16(a[i] + at + u * 32);
      };
      if (k + kDownStep <= k1) fetch(0, k);
      while (k + kDownStep <= k1) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (k + kDownStep > k1) break;
          if (k + 5 * kDownStep <= k1) fetch(y ^ 1, k + 4 * kDownStep);
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
              for (int m = 0; m < MT; ++m)
                acc[i][m] = mfma_few(av[y][i][u], xv[y][m][u], acc[i][m]);
          k += 4 * kDownStep;
        }
      }
      for (; k < k1; k += 32) {
        const bool in = k + g * 8 < k1;
        i32x4 xv[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) xv[m] = in ? load16(x[m] + k) : i32x4{};
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const i32x4 av = in ? load16(a[i] + k) : i32x4{};
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[i][m] = mfma_few(av, xv[m], acc[i][m]);
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) sums[wave][i * MT + m][lane] = acc[i][m];
      __syncthreads();
#pragma unroll
      for (int m = 0; m < MT; ++m)
        for (int i = 0; i < RT; ++i) {
          if (((i * MT + m) & 3) != wave) continue;
          const f32x4 s = ((sums[0][i * MT + m][lane] + sums[1][i * MT + m][lane]) +
                           (sums[2][i * MT + m][lane] + sums[3][i * MT + m][lane])) * scale;
          const int o = q + i * 16 + 4 * g;
          if (id[m] == ad && o < p.rank)
            *reinterpret_cast<f32x4*>(p.v + ((size_t)blockIdx.z * p.rows + row[m]) * p.rank + o) = s;
        }
      __syncthreads();
    }
  }
}

// y = the sum of the product's parts, in order, and the rows' adapters: four
// outputs to a thread.
template <bool kBF16>
__global__ __launch_bounds__(kExpertThreads) void k_lora_join(TileArgs p, const float* parts) {
  const int quads = p.n / 4;
  const int64_t total = (int64_t)p.cap * quads, stride = (int64_t)gridDim.x * kExpertThreads;
  for (int64_t i = (int64_t)blockIdx.x * kExpertThreads + threadIdx.x; i < total; i += stride) {
    const int row = (int)(i / quads), n = (int)(i - (int64_t)row * quads) * 4;
    f32x4 s = {};
    for (int x = 0; x < p.splits; ++x)
      s += *reinterpret_cast<const f32x4*>(parts + ((size_t)x * p.cap + row) * p.n + n);
    float o[4] = {s[0], s[1], s[2], s[3]};
    add_adapter(p, row, n, o);
    if constexpr (kBF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + (size_t)row * p.n + n) =
          uint2{bf16x2_rne(o[0], o[1]), bf16x2_rne(o[2], o[3])};
    else
      *reinterpret_cast<f32x4*>(static_cast<float*>(p.y) + (size_t)row * p.n + n) =
          f32x4{o[0], o[1], o[2], o[3]};
  }
}

// How a call of these sizes runs, and what it keeps in the workspace.
struct Shape {
  int down_parts;  // parts of the reduction that v is summed in
  bool few;        // k_bf16_few
  int tile_rows;   // else, of a tile
  int splits, split_stages;  // and parts of the product's reduction
  size_t v, parts;           // floats
};

Shape shape_of(const mb_lora_params& p) {
  Shape s = {};
  // few rows would leave most CUs idle: more parts
  const int blocks = (p.n_rows + 15) / 16, turns = (p.k_in + 4 * kDownStep - 1) / (4 * kDownStep);
  s.down_parts = blocks >= 64 ? 1 : std::min(turns, 4);
  s.v = (size_t)s.down_parts * p.n_rows * p.rank;
  s.few = p.n_rows <= 16;
  const int64_t columns = (p.n_out + kTileN - 1) / kTileN;
  s.tile_rows = p.n_rows > 128 && (p.n_rows + 255) / 256 * columns >= kCus / 16 ? 256 : 128;
  const int64_t tiles = std::max<int64_t>(1, (p.n_rows + s.tile_rows - 1) / s.tile_rows * columns);
  const int stages = (p.k_in + 63) / 64;
  // parts of at least four stages, as many as the CUs take at once
  const int most = std::max<int>(1, std::min<int64_t>(stages / 4, kCus / tiles));
  s.split_stages = (stages + most - 1) / most;
  s.splits = (stages + s.split_stages - 1) / s.split_stages;
  s.parts = s.few || s.splits == 1 ? 0 : (size_t)s.splits * p.n_rows * p.n_out;
  return s;
}

}  // namespace

size_t lora_workspace_floats(const mb_lora_params& p) {
  const Shape s = shape_of(p);
  return (s.v + 63) / 64 * 64 + s.parts;
}

hipError_t launch_project_lora(const mb_lora_params& q, const uint16_t* x, const uint16_t* w,
                               const uint16_t* a, const uint16_t* b, const float* scale,
                               const int32_t* adapter, float* ws, void* y, hipStream_t st) {
  if (q.n_rows == 0) return hipSuccess;
  const Shape s = shape_of(q);
  const dim3 block(kExpertThreads);
  TileArgs p = {};
  p.a = x, p.w = w, p.y = y, p.cap = q.n_rows, p.n = q.n_out, p.k = q.k_in;
  p.E = 1, p.v = ws, p.b = b, p.adapter = adapter, p.rank = q.rank, p.L = q.n_adapters;
  p.parts = s.down_parts, p.splits = s.splits, p.split_stages = s.split_stages;
  float* const parts = ws + (s.v + 63) / 64 * 64;
  const DownArgs d = {x, a, scale, adapter, ws, q.n_rows, q.k_in, q.rank, q.n_adapters, p.parts};
  const int blocks = (q.n_rows + 15) / 16;
  if (s.down_parts > 1 || blocks < kCus) {
    const dim3 grid(blocks, blocks >= 64 ? 4 : 16, s.down_parts);
    if (q.rank <= 16)
      hipLaunchKernelGGL((k_lora_down<1, 1>), grid, block, 0, st, d);
    else
      hipLaunchKernelGGL((k_lora_down<2, 1>), grid, block, 0, st, d);
  } else {
    const dim3 grid((blocks + 3) / 4);
    if (q.rank <= 16)
      hipLaunchKernelGGL((k_lora_down<1, 4>), grid, block, 0, st, d);
    else
      hipLaunchKernelGGL((k_lora_down<2, 4>), grid, block, 0, st, d);
  }
  hipError_t rc = hipGetLastError();
  if (rc != hipSuccess) return rc;
  const bool bf16 = q.dtype_out == MB_BF16;
  const dim3 cus(kCus);
  if (s.few) {
    const dim3 grid(std::min((q.n_out + 15) / 16, kFewGroups)), wide(512);
    if (bf16)
      hipLaunchKernelGGL((k_bf16_few<kTileLora, true, 8, 8>), grid, wide, 0, st, p);
    else
      hipLaunchKernelGGL((k_bf16_few<kTileLora, false, 8, 8>), grid, wide, 0, st, p);
  } else if (s.splits > 1) {
    p.y = parts;
    if (s.tile_rows == 256)
      hipLaunchKernelGGL((k_bf16_tile<kTileSplit, false, 4>), cus, block, 0, st, p);
    else
      hipLaunchKernelGGL((k_bf16_tile<kTileSplit, false, 2>), cus, block, 0, st, p);
    rc = hipGetLastError();
    if (rc != hipSuccess) return rc;
    p.y = y;
    const int64_t quads = (int64_t)q.n_rows * q.n_out / 4;
    const dim3 grid((unsigned)std::min<int64_t>((quads + 255) / 256, 4 * kFewGroups));
    if (bf16)
      hipLaunchKernelGGL((k_lora_join<true>), grid, block, 0, st, p, parts);
    else
      hipLaunchKernelGGL((k_lora_join<false>), grid, block, 0, st, p, parts);
  } else if (s.tile_rows == 256) {
    if (bf16)
      hipLaunchKernelGGL((k_bf16_tile<kTileLora, true, 4>), cus, block, 0, st, p);
    else
      hipLaunchKernelGGL((k_bf16_tile<kTileLora, false, 4>), cus, block, 0, st, p);
  } else {
    if (bf16)
      hipLaunchKernelGGL((k_bf16_tile<kTileLora, true, 2>), cus, block, 0, st, p);
    else
      hipLaunchKernelGGL((k_bf16_tile<kTileLora, false, 2>), cus, block, 0, st, p);
  }
  return hipGetLastError();
}

}  // namespace mb
