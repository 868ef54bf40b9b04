// router.hip — router logits to expert ids and gate weights (mb_route).
//
// The choice is exact: choice values are formed and compared in binary64,
// so that it is the one the definition makes on the given logits and biases
// (two values closer than binary64 resolves count as tied). Where the order
// of the choice values is the order of the logits (no bias, group scores
// that are a maximum), the logits themselves are compared.
#include <math.h>

#include "mb_internal.h"
#include "wave.h"

namespace mb {
namespace {

constexpr int kRouteWaves = 4;

template <bool kBF16>
__device__ __forceinline__ float load_logit(const void* p, size_t i) {
  if constexpr (kBF16)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else
    return static_cast<const float*>(p)[i];
}

// Logit or bias that masks its expert.
__device__ __forceinline__ bool masks(float v) { return !(v > -INFINITY); }

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  int N, E, K, G, top_groups, group_top;
  int sigmoid, renorm;
  float scale;
};

// Gate weights of a token, lane j < K holding the j-th chosen id and whether
// it is masked; `top` and `z`: the token's largest unmasked logit and
// sum exp(l - top) (softmax without renormalisation only). Both score
// functions are shifted by the largest chosen logit before they are divided
// by their sum, so that rows whose scores underflow keep their ratios.
template <bool kBF16>
__device__ void store_weights(const RouteArgs& a, size_t t, int lane, int id, bool masked,
                              double top, double z) {
  const float lj = lane < a.K ? load_logit<kBF16>(a.logits, t * a.E + id) : 0.0f;
  const bool live = lane < a.K && !masked;
  double e = 0.0;
  if (a.sigmoid) {
    const float neg = live ? fminf(lj, 0.0f) : -INFINITY;
    const float c = a.renorm ? wave_max_f32(neg) : 0.0f;
    if (live) e = exp((double)neg - (double)c) / (1.0 + exp(-fabs((double)lj)));
  } else {
    double c = top;
    if (a.renorm) c = wave_max_f32(live ? lj : -INFINITY);
    if (live) e = lj == c ? 1.0 : exp((double)lj - c);
  }
  const double norm = a.renorm ? wave_sum_f64(e) : a.sigmoid ? 1.0 : z;
  if (lane < a.K) {
    a.ids[t * a.K + lane] = id;
    a.w[t * a.K + lane] = norm > 0.0 ? (float)(e / norm * (double)a.scale) : 0.0f;
  }
}

// One token by one wave in binary64, any sizes: lane holds experts
// i*64 + lane, i < V. `arr`: LDS for V*64 doubles of this wave.
template <bool kBF16, int V>
__device__ void route_exact(const RouteArgs& a, size_t t, int lane, double* arr) {
  constexpr int kTaken = INT32_MAX;
  const bool grouped = a.top_groups < a.G;
  const bool by_logit = !a.bias && (!grouped || a.group_top == 1);
  float l[V];
  double c[V];
  int id[V];  // expert id; past all ids once closed or taken
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    id[i] = e < a.E ? e : kTaken;
    l[i] = e < a.E ? load_logit<kBF16>(a.logits, t * a.E + e) : -INFINITY;
    if (masks(l[i])) l[i] = -INFINITY;
    mx = fmaxf(mx, l[i]);
  }
  double z = 0.0;
  if (!a.sigmoid && (!a.renorm || !by_logit)) {
    mx = wave_max_f32(mx);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (l[i] > -INFINITY) z += l[i] == mx ? 1.0 : exp((double)l[i] - (double)mx);
    z = wave_sum_f64(z);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = (double)l[i];
    if (!by_logit && l[i] > -INFINITY) {
      if (a.sigmoid)
        c[i] = l[i] >= 0.0f ? 1.0 / (1.0 + exp(-(double)l[i]))
                            : exp((double)l[i]) / (1.0 + exp((double)l[i]));
      else
        c[i] = (l[i] == mx ? 1.0 : exp((double)l[i] - (double)mx)) / z;
      if (a.bias) {
        const float b = a.bias[i * 64 + lane];
        c[i] = masks(b) ? -INFINITY : c[i] + (double)b;
      }
    }
  }
  if (grouped) {
    const int size = a.E / a.G;
#pragma unroll
    for (int i = 0; i < V; ++i) arr[i * 64 + lane] = c[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    double t1 = -INFINITY, t2 = -INFINITY;
    if (lane < a.G) {
      for (int i = 0; i < size; ++i) {
        const double v = arr[lane * size + i];
        t2 = fmax(t2, fmin(t1, v));
        t1 = fmax(t1, v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    double s = t1;
    if (a.group_top == 2) s = t2 > -INFINITY ? t1 + t2 : -INFINITY;
    int above = 0;  // groups ahead of this lane's
    for (int g = 0; g < a.G; ++g) {
      const double o = __shfl(s, g);
      above += o > s || (o == s && g < lane);
    }
    const uint64_t open = ballot64(lane < a.G && above < a.top_groups);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      if (e < a.E && !((open >> (e / size)) & 1)) {
        id[i] = kTaken;
        c[i] = -INFINITY;
      }
    }
  }
  int mine = 0;
  bool masked = false;
  for (int k = 0; k < a.K; ++k) {
    double bc = -INFINITY;
    int bid = kTaken;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c[i] > bc || (c[i] == bc && id[i] < bid)) bc = c[i], bid = id[i];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double oc = __shfl_xor(bc, m);
      const int oid = __shfl_xor(bid, m);
      if (oc > bc || (oc == bc && oid < bid)) bc = oc, bid = oid;
    }
    if (lane == k) mine = bid, masked = !(bc > -INFINITY);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (id[i] == bid) id[i] = kTaken, c[i] = -INFINITY;
  }
  store_weights<kBF16>(a, t, lane, mine, masked, mx, z);
}

template <bool kBF16, int V>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route(RouteArgs a) {
  __shared__ double arr[kRouteWaves][V * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const size_t t = (size_t)blockIdx.x * kRouteWaves + wave;
  if (t >= (size_t)a.N) return;
  route_exact<kBF16, V>(a, t, lane, arr[wave]);
}

template <bool kBF16>
void launch_route_t(const RouteArgs& a, hipStream_t st) {
  const dim3 grid((a.N + kRouteWaves - 1) / kRouteWaves), block(64 * kRouteWaves);
  const int v = (a.E + 63) / 64;
  if (v <= 1)
    hipLaunchKernelGGL((k_route<kBF16, 1>), grid, block, 0, st, a);
  else if (v <= 4)
    hipLaunchKernelGGL((k_route<kBF16, 4>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_route<kBF16, 16>), grid, block, 0, st, a);
}

}  // namespace

hipError_t launch_route(const mb_route_params& p, const void* logits, const float* bias,
                        int32_t* ids, float* w, hipStream_t st) {
  if (p.n_tokens == 0) return hipSuccess;
  const RouteArgs a = {logits,     bias,           ids,
                       w,          p.n_tokens,     p.n_experts,
                       p.top_k,    p.n_groups,     p.top_groups,
                       p.group_top, p.score == MB_SCORE_SIGMOID, p.renorm != 0,
                       p.scale};
  if (p.dtype == MB_BF16)
    launch_route_t<true>(a, st);
  else
    launch_route_t<false>(a, st);
  return hipGetLastError();
}

}  // namespace mb
