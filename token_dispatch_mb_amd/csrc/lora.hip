// lora.hip — a projection with the low-rank adapters of many requests beside
// it (mb_project_lora).
//
//   y[t] = x[t] w^T + v[t] b_a^T,  v[t] = scale_a x[t] a_a^T,  a = adapter[t]
//
// k_lora_down makes v, in binary32; the product then goes on over the ranks
// of the adapters among a tile's rows, so that w and y are passed once. 16384
// rows, 7168 x 7168, rank 32: 0.09 to 0.11 and 1.35 to 1.4 ms, 1.17 PFLOP/s in
// all (without any adapter the same: the matrix unit's power and the tiles' ends
// bound it). Rows whose adapters differ within 32 rows compute one after the
// other, each waiting for its own loads: 4096 rows of 64 adapters in turn, 4096 x
// 4096, rank 16 0.44 ms, in runs 0.14. 64
// rows with an adapter each: 8, 23 and 9 us for v, the product in nine parts
// (4.4 TB/s of w) and their sum, bound by the latency of three short kernels.
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

// v of 16 rows and 16 RT ranks, of one of their adapters or of one after the
// other: workgroup (x, y, z) takes the row block x, adapters y, y + gridDim.y,
// ... in the order of their numbers, and part z of the reduction. Its four
// waves take 128 elements by turns, the next turn's on their way while this
// one's are multiplied, and add up in LDS. Rows without an adapter are not
// written (nothing reads them).
//
// Bound by the reading of x and of the adapters, which every row block passes
// again, from the caches: 16384 rows of 7168 elements in 54, 95 and 178 us at
// rank 16, 32 and 64 (4.3, 2.5 TB/s of x). 64 rows to a workgroup pass the
// adapters a quarter as often and took 65, 79 and 152 us, and at 4096 rows,
// where too few workgroups are left, 64, 77 and 224 us for 28, 40 and 77.
template <int RT>
__global__ __launch_bounds__(kExpertThreads) void k_lora_down(DownArgs p) {
  constexpr int U = kDownStep / 32;
  __shared__ f32x4 sums[4][RT][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int row = blockIdx.x * 16 + r, at = min(row, p.rows - 1);
  int id = p.adapter[at];
  if ((unsigned)id >= (unsigned)p.L || row >= p.rows) id = INT32_MAX;
  const uint16_t* x = p.x + (int64_t)at * p.k + g * 8;
  // part z: whole turns of four waves
  const int turns = (p.k + 4 * kDownStep - 1) / (4 * kDownStep);
  const int each = (turns + p.parts - 1) / p.parts;
  const int k0 = min((int)blockIdx.z * each * 4 * kDownStep, p.k);
  const int k1 = min(k0 + each * 4 * kDownStep, p.k);
  int ad = -1;
  for (int j = 0;; ++j) {
    ad = wave_min_i32(id > ad ? id : INT32_MAX);
    if (ad == INT32_MAX) break;
    if (j % gridDim.y != blockIdx.y) continue;
    const float scale = p.scale[ad];
    for (int q = 0; q < p.rank; q += 16 * RT) {
      const uint16_t* a[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
        a[i] = p.a + ((int64_t)ad * p.rank + min(q + i * 16 + r, p.rank - 1)) * p.k + g * 8;
      f32x4 acc[RT] = {};
      int k = k0 + wave * kDownStep;
      i32x4 xv[2][U], av[2][RT][U];
      auto fetch = [&](int to, int at) {
#pragma unroll
        for (int u = 0; u < U; ++u) xv[to][u] = load16(x + at + u * 32);
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
            for (int i = 0; i < RT; ++i) acc[i] = mfma_few(av[y][i][u], xv[y][u], acc[i]);
          k += 4 * kDownStep;
        }
      }
      for (; k < k1; k += 32) {
        const bool in = k + g * 8 < k1;
        const i32x4 xs = in ? load16(x + k) : i32x4{};
#pragma unroll
        for (int i = 0; i < RT; ++i)
          acc[i] = mfma_few(in ? load16(a[i] + k) : i32x4{}, xs, acc[i]);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) sums[wave][i][lane] = acc[i];
      __syncthreads();
      if (wave < RT) {
        const f32x4 s = ((sums[0][wave][lane] + sums[1][wave][lane]) +
                         (sums[2][wave][lane] + sums[3][wave][lane])) * scale;
        const int o = q + wave * 16 + 4 * g;
        if (id == ad && o < p.rank)
          *reinterpret_cast<f32x4*>(p.v + ((size_t)blockIdx.z * p.rows + row) * p.rank + o) = s;
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

int64_t tiles_of(const mb_lora_params& p, int rows) {
  return ((int64_t)p.n_rows + rows - 1) / rows * ((p.n_out + kTileN - 1) / kTileN);
}

// In eighths of a microsecond, roughly: a stage of a 128-row tile takes eight,
// of a 256-row tile kLongTile; where there are parts, a launch takes 3 us and
// their sums are written and read back at 5 TB/s.
int64_t tiles_cost(const mb_lora_params& p, int rows, int splits) {
  const int64_t tiles = tiles_of(p, rows);
  const int stages = ((p.k_in + 63) / 64 + splits - 1) / splits;
  const int64_t cost = (tiles * splits + kCus - 1) / kCus * stages * (rows == 256 ? kLongTile : 8);
  return cost + (splits > 1 ? 24 + (int64_t)splits * p.n_rows * p.n_out / 80000 : 0);
}

Shape shape_of(const mb_lora_params& p) {
  Shape s = {};
  // few rows would leave most CUs idle: more parts (64 rows of 7168 elements,
  // rank 16: 15.5 us in one part, 9.6 in four; 4096 rows: 28 and 20, but the
  // product reads v four times)
  const int blocks = (p.n_rows + 15) / 16, turns = (p.k_in + 4 * kDownStep - 1) / (4 * kDownStep);
  s.down_parts = blocks >= 64 ? 1 : std::min(turns, 4);
  s.v = (size_t)s.down_parts * p.n_rows * p.rank;
  // A block of rows, or no more than a 16 x 16 tile to a CU, straight from
  // memory, us, against the tiles: 16 rows, n_out = k_in = 4096 19, 25 (24
  // rows: 28, 27); k_in = 7168: 240 rows, n_out = 256 28, 34; 4000 rows, 8 42,
  // 51; 64 rows, 1024 23, 31. Two tiles to a CU (64 rows, 2048): 37, 31, though of
  // short reductions they are the faster too (k_in = 1024: 11, 21).
  s.few = p.n_rows <= 16 || (int64_t)blocks * ((p.n_out + 15) / 16) <= kCus;
  // else the cheapest of both tiles and of up to as many parts as the CUs take
  // at once, of at least four stages. n_out = k_in = 7168, the best of 128-row
  // tiles against 256-row tiles, us: 384 rows 74, 85; 1024 rows 123, 151;
  // 4096 rows 486, 473; of one part against several: 512 rows 121, 87; 2048 x
  // 2048 x 2048: 51, 58.
  const int stages = (p.k_in + 63) / 64;
  int64_t best = INT64_MAX;
  for (int rows = 128; rows <= 256; rows += 128) {
    const int64_t tiles = std::max<int64_t>(1, tiles_of(p, rows));
    const int most = std::max<int>(1, std::min<int64_t>(stages / 4, kCus / tiles));
    for (int splits = 1; splits <= most; ++splits) {
      const int64_t cost = tiles_cost(p, rows, splits);
      if (cost >= best) continue;
      best = cost;
      s.tile_rows = rows;
      s.split_stages = (stages + splits - 1) / splits;
    }
  }
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
  // (a block's rows have up to 16 adapters; in long batches, mostly one)
  const dim3 down(blocks, blocks >= 64 ? 4 : 16, s.down_parts);
  if (q.rank <= 16)
    hipLaunchKernelGGL((k_lora_down<1>), down, block, 0, st, d);
  else
    hipLaunchKernelGGL((k_lora_down<2>), down, block, 0, st, d);
  hipError_t rc = hipGetLastError();
  if (rc != hipSuccess) return rc;
  const bool bf16 = q.dtype_out == MB_BF16;
  const dim3 cus(kCus);
  if (s.few) {
    const dim3 grid((unsigned)std::min<int64_t>((int64_t)blocks * ((q.n_out + 15) / 16), kFewGroups));
    const dim3 wide(512);
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
