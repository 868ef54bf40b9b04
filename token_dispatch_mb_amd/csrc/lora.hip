// lora.hip — a projection with the low-rank adapters of many requests beside
// it (mb_project_lora).
//
//   y[t] = x[t] w^T + v[t] b_a^T,  v[t] = scale_a x[t] a_a^T,  a = adapter[t]
//
// k_lora_down makes v, in binary32; the product then goes on over the ranks
// of the adapters among a tile's rows, so that w and y are passed once.
#include "bf16_tile.h"

namespace mb {
namespace {

constexpr int kFewGroups = 2048;

struct DownArgs {
  const uint16_t* x;
  const uint16_t* a;  // [L][rank][k]
  const float* scale;
  const int32_t* adapter;
  float* v;  // [parts][rows][rank]
  int rows, k, rank, L, parts;
};

// v of 16 rows and 16 RT ranks of one of their adapters, or of one after the
// other: workgroup (x, y, z) takes the row block x, adapters y, y + gridDim.y,
// ... in the order of their numbers, and part z of the reduction. Its four
// waves take 128 elements by turns and add up in LDS. Rows without an adapter
// are not written (nothing reads them).
template <int RT>
__global__ __launch_bounds__(kExpertThreads) void k_lora_down(DownArgs p) {
  constexpr int U = kFewStep / 32;
  __shared__ f32x4 sums[4][RT][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int row = blockIdx.x * 16 + r;
  const int at = min(row, p.rows - 1);
  int id = p.adapter[at];
  if ((unsigned)id >= (unsigned)p.L || row >= p.rows) id = INT32_MAX;
  // part z: whole turns of four waves
  const int turns = (p.k + 4 * kFewStep - 1) / (4 * kFewStep);
  const int each = (turns + p.parts - 1) / p.parts;
  const int k0 = min(blockIdx.z * each * 4 * kFewStep, (unsigned)p.k);
  const int k1 = min(k0 + each * 4 * kFewStep, p.k);
  const uint16_t* x = p.x + (int64_t)at * p.k + g * 8;
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
      int k = k0 + wave * kFewStep;
      for (; k + kFewStep <= k1; k += 4 * kFewStep) {
        i32x4 xv[U], av[RT][U];
#pragma unroll
        for (int u = 0; u < U; ++u) xv[u] = load16(x + k + u * 32);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int u = 0; u < U; ++u) av[i][u] = load16(a[i] + k + u * 32);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[i] = mfma_few(av[i][u], xv[u], acc[i]);
      }
      for (; k < k1; k += 32) {
        const bool in = k + g * 8 < k1;
        const i32x4 xv = in ? load16(x + k) : i32x4{};
#pragma unroll
        for (int i = 0; i < RT; ++i)
          acc[i] = mfma_few(in ? load16(a[i] + k) : i32x4{}, xv, acc[i]);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) sums[wave][i][lane] = acc[i];
      __syncthreads();
      for (int i = wave; i < RT; i += 4) {
        const f32x4 s = ((sums[0][i][lane] + sums[1][i][lane]) +
                         (sums[2][i][lane] + sums[3][i][lane])) * scale;
        const int o = q + i * 16 + 4 * g;
        if (id == ad && o < p.rank)
          *reinterpret_cast<f32x4*>(p.v + ((size_t)blockIdx.z * p.rows + row) * p.rank + o) = s;
      }
      __syncthreads();
    }
  }
}

}  // namespace

// Parts of the reduction that v is summed in: more where few rows would
// leave most CUs idle.
int lora_parts(const mb_lora_params& p) {
  const int blocks = (p.n_rows + 15) / 16, turns = (p.k_in + 4 * kFewStep - 1) / (4 * kFewStep);
  return blocks >= 64 ? 1 : min(turns, 4);
}

hipError_t launch_project_lora(const mb_lora_params& q, const uint16_t* x, const uint16_t* w,
                               const uint16_t* a, const uint16_t* b, const float* scale,
                               const int32_t* adapter, float* v, void* y, hipStream_t st) {
  if (q.n_rows == 0) return hipSuccess;
  const dim3 block(kExpertThreads);
  const int blocks = (q.n_rows + 15) / 16;
  TileArgs p = {};
  p.a = x, p.w = w, p.y = y, p.cap = q.n_rows, p.n = q.n_out, p.k = q.k_in;
  p.E = 1, p.v = v, p.b = b, p.adapter = adapter, p.rank = q.rank, p.L = q.n_adapters;
  p.parts = lora_parts(q);
  if (q.n_adapters > 0) {
    const DownArgs d = {x, a, scale, adapter, v, q.n_rows, q.k_in, q.rank, q.n_adapters, p.parts};
    const dim3 grid(blocks, blocks >= 64 ? 1 : 16, p.parts);
    if (q.rank <= 16)
      hipLaunchKernelGGL((k_lora_down<1>), grid, block, 0, st, d);
    else
      hipLaunchKernelGGL((k_lora_down<2>), grid, block, 0, st, d);
    const hipError_t rc = hipGetLastError();
    if (rc != hipSuccess) return rc;
  }
  const bool bf16 = q.dtype_out == MB_BF16;
#define MB_L(KERNEL, X, GRID)                                                       \
  do {                                                                              \
    if (bf16)                                                                       \
      hipLaunchKernelGGL((KERNEL<kTileLora, true, X>), GRID, block, 0, st, p);      \
    else                                                                            \
      hipLaunchKernelGGL((KERNEL<kTileLora, false, X>), GRID, block, 0, st, p);     \
  } while (0)
  if (q.n_rows <= 16)
    MB_L(k_bf16_few, 1, dim3(kFewGroups));
  else if (q.n_rows <= 64)
    MB_L(k_bf16_few, 4, dim3(kFewGroups));
  else if ((int64_t)((q.n_rows + 255) / 256) * ((q.n_out + 255) / 256) >= kCus)
    MB_L(k_bf16_tile, 4, dim3(kCus));
  else
    MB_L(k_bf16_tile, 2, dim3(kCus));
#undef MB_L
  return hipGetLastError();
}

}  // namespace mb
