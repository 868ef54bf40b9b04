// router.hip — router logits to expert ids and gate weights (mb_route).
//
// The choice is exact: choice values are formed and compared in binary64
// wherever binary32 cannot tell them apart, so that it is the one the
// definition makes on the given logits and biases (two values closer than
// binary64 resolves count as tied). Where the order
// of the choice values is the order of the logits (no bias, group scores
// that are a maximum), the logits themselves are compared.
#include <math.h>

#include <type_traits>

#include "mb_internal.h"
#include "wave.h"

namespace mb {
namespace {

constexpr int kRouteWaves = 4;
constexpr int kRouteGroups = 2048;  // workgroups of one launch: eight for each CU, two to five of them at a time

template <bool kBF16>
__device__ __forceinline__ float load_logit(const void* p, size_t i) {
  if constexpr (kBF16)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else
    return static_cast<const float*>(p)[i];
}

// V consecutive logits at i, both multiples of 4.
template <bool kBF16, int V>
__device__ __forceinline__ void load_row(const void* p, size_t i, float* v) {
#pragma unroll
  for (int j = 0; j + 3 < V; j += 4) {
    if constexpr (kBF16) {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i + j);
      v[j] = __uint_as_float(u.x << 16), v[j + 1] = __uint_as_float(u.x & 0xffff0000u);
      v[j + 2] = __uint_as_float(u.y << 16), v[j + 3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + j);
      v[j] = f.x, v[j + 1] = f.y, v[j + 2] = f.z, v[j + 3] = f.w;
    }
  }
}

// Logit or bias that masks its expert.
__device__ __forceinline__ bool masks(float v) { return !(v > -INFINITY); }

template <int kCtrl>
__device__ __forceinline__ int dpp_i32(int v) {
  return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xf, 0xf, true);
}

// Float bits to integers of the same order, and back. (Sorting compares
// integers: a float maximum of bits the compiler did not compute costs two
// more instructions, in case they are a signalling NaN.)
__device__ __forceinline__ int sortable(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unsortable(int s) {
  return __int_as_float(s ^ ((s >> 31) & 0x7fffffff));
}

__device__ __forceinline__ int row_max_i32(int v) {
  v = max(v, dpp_i32<0xB1>(v));
  v = max(v, dpp_i32<0x4E>(v));
  v = max(v, dpp_i32<0x141>(v));
  return max(v, dpp_i32<0x140>(v));
}

__device__ __forceinline__ float wave_max_f32(float v) { return unsortable(wave_max_i32(sortable(v))); }

template <int kCtrl>
__device__ __forceinline__ double dpp_f64(double v) {
  return __hiloint2double(dpp_i32<kCtrl>(__double2hiint(v)), dpp_i32<kCtrl>(__double2loint(v)));
}

__device__ __forceinline__ double lane_f64(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}

__device__ __forceinline__ double wave_sum_f64(double v) {
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x141>(v);
  v += dpp_f64<0x140>(v);
  return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}

// The largest value of the wave and, among its holders, the lowest id: three
// integer reductions (high words, low words, ids).
__device__ __forceinline__ int wave_argmax(double v, int id, double& best) {
  v += 0.0;  // one zero, whatever its sign
  const int h0 = __double2hiint(v), l0 = __double2loint(v), neg = h0 >> 31;
  const int hi = h0 ^ (neg & 0x7fffffff), lo = (l0 ^ neg) ^ INT32_MIN;  // in order, as signed words
  const int mh = wave_max_i32(hi);
  const int ml = wave_max_i32(hi == mh ? lo : INT32_MIN);
  const int mneg = mh >> 31;
  best = __hiloint2double(mh ^ (mneg & 0x7fffffff), (ml ^ INT32_MIN) ^ mneg);
  return wave_min_i32(hi == mh && lo == ml ? id : INT32_MAX);
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
#pragma unroll 8
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
      const double o = lane_f64(s, g);
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
    bid = wave_argmax(bc, bid, bc);
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

// ---- four tokens to a wave, in binary32 --------------------------------------
//
// A token on a row of 16 lanes, V consecutive experts to a lane. Choice
// values become integer keys whose low bits hold the expert's place in its
// lane, so that sorting moves one register per expert; each lane sorts its
// keys once, and a round takes the largest head of the row (four DPP steps)
// and shifts the list of the lane that owned it. Everything is compared in
// binary32, which decides unless two values come closer than its rounding.
// Such neighbours among the first K + 1 are ranked by their binary64 values
// (a lane computes one); a row where that does not settle it (the last open
// and the first closed group, more candidates than K + 1, softmax scores with
// a bias, masked or infinite choices) is done again by route_exact. bf16
// logits compared as themselves have 16 free bits: their keys hold the whole
// expert id and are exact, ties included.
//
// Bound by vector instructions (about 900 for a wave's four tokens of 256
// experts: a third for scores and keys, a third for the rounds), not by the
// 6.3 TB/s its reads could have. Measured on MI355X: 131072 tokens x 256
// experts in 8 groups, fp32, sigmoid and bias: 64 us (2.2 TB/s; a wave per
// token in binary64 takes 355); without route_exact's rows, a few in 100000,
// it would be 13 us less, their one long chain being the tail. 65536 x 384,
// softmax: 31 us (3.4 TB/s). 8192 x 256, bf16: 9 us, and 16 with a row redone.

// By value: of two array elements the compiler would choose the index.
__device__ __forceinline__ int choose(bool c, int a, int b) { return c ? a : b; }

// a >= b
__device__ __forceinline__ void order(int& a, int& b) {
  const int t = max(a, b);
  b = min(a, b);
  a = t;
}

// N (a power of two) values at k, descending: odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_desc(int* k) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int j = d % p; j + d < N; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i)
          if (i + j + d < N && (i + j) / (2 * p) == (i + j + d) / (2 * p)) order(k[i + j], k[i + j + d]);
}

// The 8 largest of two descending lists of 8, descending, into a.
__device__ __forceinline__ void merge8(int* a, const int* b) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
#pragma unroll
  for (int d = 4; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) order(a[i], a[i + d]);
}

constexpr float kHuge = 3e38f;  // choice values past it are masks or infinities

// Groups of kLanes lanes of a row whose value is above this one's.
template <int kLanes, int kRor = kLanes>
__device__ __forceinline__ int groups_above(float v) {
  if constexpr (kRor == 16) {
    return 0;
  } else {
    const float o = __int_as_float(dpp_i32<0x120 + kRor>(__float_as_int(v)));
    return (o > v ? 1 : 0) + groups_above<kLanes, kRor + kLanes>(v);
  }
}

// Lanes of the row whose value comes before this one's: larger, or equal with
// a lower id.
template <int kRor>
__device__ __forceinline__ int lanes_ahead(double v, int id) {
  if constexpr (kRor == 16) {
    return 0;
  } else {
    const int o_id = dpp_i32<0x120 + kRor>(id);
    const double o = dpp_f64<0x120 + kRor>(v);
    return (o > v || (o == v && o_id < id) ? 1 : 0) + lanes_ahead<kRor + 1>(v, id);
  }
}

// KT: top K known when compiled, or 0.
template <bool kBF16, int V, bool kByLogit, bool kGrouped, int KT>
__global__ __launch_bounds__(64 * kRouteWaves) void k_route_rows(RouteArgs a, int quads) {
  const int K = KT ? KT : a.K;
  constexpr int L = V < 8 ? V : 8;  // length of a lane's list
  constexpr int VE = (V + 3) / 4;
  constexpr bool kWholeId = kBF16 && kByLogit;
  constexpr int kIdBits = V <= 1 ? 0 : V <= 2 ? 1 : V <= 4 ? 2 : V <= 8 ? 3 : V <= 16 ? 4 : 5;
  constexpr int kIdMask = (1 << kIdBits) - 1;
  constexpr float kLog2e = 1.44269504f;
  __shared__ double arr[kGrouped ? kRouteWaves : 1][kGrouped ? VE * 64 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane & 15, row = lane >> 4;
  const int e0 = q * V;
  // How far rounding may move a choice value, in units of 2^-24 (a product's
  // rounding, relative). A score s: the products in front of the exponential
  // are off by their own size, which is at most ln(1/s): 1.22 ln(1/s) with the
  // constant's error, 2.22 for softmax, where the difference to the largest
  // logit is rounded before; exponential, sum and reciprocal add 5 (the
  // instructions' own errors stay below 2 each, measured), and 54 where the
  // sum goes over a row (32 terms in line). s is unknown beside a
  // bias: at most |choice| + |bias|, and 1. (s ln(1/s) rises with s up to 1/e;
  // past it the constants cover it.) A choice value is rounded once more, and
  // cut by the place in its key.
  const float per_log2 = a.sigmoid ? 0.85f : 1.54f, fixed = a.sigmoid ? 5.0f : 54.0f;
  constexpr float kUnit = 0x1.1p-24f;  // with room for products of two errors
  constexpr float kKey = kWholeId ? 0.0f : (float)(2 << kIdBits);
  constexpr float kTiny = 0x1p-100f;  // below it the places in the keys count
  const bool whole = V % 4 == 0 && a.E == 16 * V;
  float b[V], bmax = 0.0f;
  // no lane without experts, no bias that is not a number (by logits alone
  // the masks cost less than the test for them)
  bool plain = whole && !kByLogit;
  if constexpr (!kByLogit) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      b[i] = a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
      if (masks(b[i])) b[i] = -INFINITY;
      if (fabsf(b[i]) < INFINITY) bmax = fmaxf(bmax, fabsf(b[i]));
      else plain = false;
    }
    bmax = row_max_f32(bmax);
    plain = ballot64(!plain) == 0;
  }
  // the part of a score whose choice value is `v` in magnitude
  auto score_error = [&](float v) {
    const float most = fminf(v + bmax + kTiny, 1.0f);
    return most * (per_log2 * (float)(127 - (int)(__float_as_uint(most) >> 23)) + fixed);
  };
  // Logits of quad w; rows past the last token repeat it (and store nothing).
  // Those of the next quad are fetched while the rounds of one run.
  float c[V];
  auto fetch = [&](int w) {
    const size_t i = (size_t)min(w * 4 + row, a.N - 1) * a.E + e0;
    if (whole) {
      load_row<kBF16, V>(a.logits, i, c);
    } else if (V % 4 == 0 && (a.E & 3) == 0) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        c[j] = c[j + 1] = c[j + 2] = c[j + 3] = -INFINITY;
        if (e0 + j < a.E) load_row<kBF16, 4>(a.logits, i + j, c + j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] = e0 + j < a.E ? load_logit<kBF16>(a.logits, i + j) : -INFINITY;
    }
  };
  int w = blockIdx.x * kRouteWaves + wave;
  const int stride = gridDim.x * kRouteWaves;
  if (w < quads) fetch(w);
  for (; w < quads; w += stride) {
    const int t = min(w * 4 + row, a.N - 1);
    const size_t at = (size_t)t * a.E;
    float mx = -INFINITY, z = 0.0f;
    int k[V];
    // choice values and their keys; kMasks: some may be masked or infinite
    auto score = [&](auto masks_) {
      constexpr bool kMasks = decltype(masks_)::value;
      if constexpr (kMasks) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = c[i] > -INFINITY ? c[i] : -INFINITY;  // NaN masks too
      }
      if (!a.sigmoid && (!kByLogit || !a.renorm)) {
#pragma unroll
        for (int i = 0; i < V; ++i) mx = fmaxf(mx, c[i]);
        mx = row_max_f32(mx);
#pragma unroll
        for (int i = 0; i < V; ++i) z += __builtin_amdgcn_exp2f((c[i] - mx) * kLog2e);
        z = row_sum_f32(z);
      }
      if constexpr (!kByLogit) {
        if (a.sigmoid) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-c[i] * kLog2e));
            c[i] = !kMasks || c[i] > -INFINITY ? s + b[i] : -INFINITY;
          }
        } else {
          const float rz = 1.0f / z;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float s = __builtin_amdgcn_exp2f((c[i] - mx) * kLog2e) * rz;
            c[i] = !kMasks || c[i] > -INFINITY ? s + b[i] : -INFINITY;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float v = c[i] + 0.0f;  // one zero, whatever its sign
        k[i] = sortable(kMasks ? __builtin_amdgcn_fmed3f(v, -kHuge, kHuge) : v);
      }
    };
    float probe = 0.0f;  // NaN if a logit is no number
    if (plain) {
#pragma unroll
      for (int i = 0; i < V; ++i) probe = fmaf(c[i], 0.0f, probe);
    }
    if (plain && ballot64(probe != probe) == 0)
      score(std::false_type());
    else
      score(std::true_type());
    bool again = !(mx < INFINITY) || (!a.sigmoid && !(z < INFINITY));
    bool open = true;
    if constexpr (kGrouped) {
      const int lanes = a.E / a.G / V;  // of a group: 1, 2, 4 or 8
      int t1 = INT32_MIN, t2 = INT32_MIN;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t2 = max(t2, min(t1, k[i]));
        t1 = max(t1, k[i]);
      }
      auto join = [&](int o1, int o2) {
        t2 = max(min(t1, o1), max(t2, o2));
        t1 = max(t1, o1);
      };
      if (lanes > 1) join(dpp_i32<0xB1>(t1), dpp_i32<0xB1>(t2));
      if (lanes > 2) join(dpp_i32<0x4E>(t1), dpp_i32<0x4E>(t2));
      if (lanes > 4) join(dpp_i32<0x141>(t1), dpp_i32<0x141>(t2));
      const float f1 = unsortable(t1), f2 = unsortable(t2);
      // with a masked second best the sum is -inf
      const float gs = a.group_top == 1 ? f1 : f2 > -kHuge ? f1 + f2 : -kHuge;
      const int above = lanes == 1   ? groups_above<1>(gs)
                        : lanes == 2 ? groups_above<2>(gs)
                        : lanes == 4 ? groups_above<4>(gs)
                                     : groups_above<8>(gs);
      open = above < a.top_groups;
      const uint32_t seg = (uint32_t)(ballot64(open) >> (row * 16)) & 0xffffu;
      // what the exact score may be at least and at most (maxima of logits are exact)
      float off = 0.0f;
      if constexpr (!kByLogit) {
        const bool two = a.group_top == 2;
        const float sum = fabsf(f1) + (two ? fabsf(f2) : 0.0f);
        off = two ? 2.0f * score_error(0.5f * sum) : score_error(sum);
        off = kUnit * off + kUnit * sum + 2.0f * kUnit * fabsf(gs);
      }
      const float low = unsortable(~row_max_i32(open ? ~sortable(gs - off) : INT32_MIN));
      const float high = unsortable(row_max_i32(open ? INT32_MIN : sortable(gs + off)));
      // unless exactly top_groups groups are ahead of the rest by more than
      // rounding, and their scores are numbers
      again |= __popc(seg) != a.top_groups * lanes || !(fabsf(low) < 0.99f * kHuge) || !(low > high);
    }
    // the low bits: larger for the lower id
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (kWholeId)
        k[i] = (k[i] & ~0xffff) | (0xffff - (e0 + i));
      else
        k[i] = (k[i] & ~kIdMask) | (kIdMask - i);
      if (!whole && e0 + i >= a.E) k[i] = INT32_MIN;
    }
    if (w + stride < quads) fetch(w + stride);
    if constexpr (V <= 8) {
      sort_desc<V>(k);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 8) sort_desc<8>(k + i);
#pragma unroll
      for (int i = 8; i < V; i += 8) merge8(k, k + i);
    }
    if constexpr (kGrouped) {
#pragma unroll
      for (int i = 0; i < L; ++i) k[i] = choose(open, k[i], INT32_MIN);
    }
    // round j: lane j notes the j-th largest key and the lane it came from
    int mine = INT32_MIN, from = 0, taken = 0;
    auto round = [&](int j) {
      const int m = row_max_i32(k[0]);
      bool win = k[0] == m;
      if constexpr (!kWholeId) {
        const int lowest = __ffs((uint32_t)(ballot64(win) >> (row * 16)) & 0xffffu) - 1;
        win = q == lowest;  // equal keys one at a time
        if (q == j) from = lowest;
      }
      if (q == j) mine = m;
      taken += win;
#pragma unroll
      for (int i = 0; i + 1 < L; ++i) k[i] = choose(win, k[i + 1], k[i]);
      k[L - 1] = choose(win, INT32_MIN, k[L - 1]);
    };
    if constexpr (KT > 0) {
#pragma unroll
      for (int j = 0; j < (kWholeId ? KT : KT + 2); ++j) round(j);
    } else {
      const int rounds = kWholeId ? K : K + 2;
      for (int j = 0; j < rounds; ++j) round(j);
    }
    const float value = unsortable(mine);
    again |= (V > L && taken >= L) || (q < K && !(fabsf(value) < 0.99f * kHuge));
    int id = 0;
    if constexpr (kWholeId) {
      if (q < K) id = 0xffff - (mine & 0xffff);
    } else {
      if (q <= K && mine != INT32_MIN) id = from * V + kIdMask - (mine & kIdMask);
      // Neighbours too close to tell apart, among the first K + 1: those are
      // put in order by their exact values, unless more may belong with them.
      // (NaN stands for no key at all: nothing is close to it.)
      const float next = unsortable(dpp_i32<0x101>(mine));  // row_shl 1
      const float mag = fabsf(value), off = kByLogit ? 0.0f : score_error(mag);
      const bool close = q <= K && value - next <= 2 * kUnit * (off + kKey * (mag + kTiny));
      const uint32_t seg = (uint32_t)(ballot64(close) >> (row * 16)) & 0xffffu;
      const bool near = (seg & ((1u << K) - 1u)) != 0;
      again |= near && (((seg >> (K - 1)) & 3u) == 3u || (!kByLogit && !a.sigmoid));
      if (ballot64(near && !again) != 0) {
        double d = -INFINITY;
        int key = q <= K ? id : a.E + q;
        if (q <= K && value > -0.99f * kHuge) {
          d = load_logit<kBF16>(a.logits, at + id);
          if constexpr (!kByLogit) d = 1.0 / (1.0 + exp(-d)) + (a.bias ? (double)a.bias[id] : 0.0);
        }
        const int place = lanes_ahead<1>(d, key);
        const int moved = __builtin_amdgcn_ds_permute((row * 16 + place) * 4, id);
        if (q < K) id = moved;
      }
    }
    const uint64_t redo = ballot64(again);
    const bool ours = q < K && !((redo >> (row * 16)) & 0xffffu);
    if (!ours) id = 0;
    const float l = load_logit<kBF16>(a.logits, at + id);
    float e, norm = 1.0f;
    if (a.sigmoid) {
      const float neg = fminf(l, 0.0f);
      const float shift = a.renorm ? row_max_f32(ours ? neg : -INFINITY) : 0.0f;
      e = expf(neg - shift) / (1.0f + expf(-fabsf(l)));
    } else {
      e = expf(l - (a.renorm ? row_max_f32(ours ? l : -INFINITY) : mx));
      norm = z;
    }
    if (a.renorm) norm = row_sum_f32(ours ? e : 0.0f);
    if (ours && w * 4 + row < a.N) {
      a.ids[(size_t)t * K + q] = id;
      a.w[(size_t)t * K + q] = e / norm * a.scale;
    }
    for (uint64_t left = redo; left;) {
      const int r = __builtin_ctzll(left) >> 4;
      left &= ~(0xffffull << (r * 16));
      if (w * 4 + r < a.N) route_exact<kBF16, VE>(a, (size_t)w * 4 + r, lane, arr[kGrouped ? wave : 0]);
    }
  }
}

// Whether k_route_rows<V> takes these sizes: groups must be whole lanes, and
// are found by a lane's place alone, so that the row must be full of them. (Other
// sizes run in binary64, about five times slower: 131072 x 256 by k_route 355 us,
// 64 here.)
bool rows_fit(const RouteArgs& a, int V, bool grouped) {
  if (a.K > 14) return false;
  if (!grouped) return true;
  const int size = a.E / a.G;
  return a.E == 16 * V && size % V == 0;
}

template <bool kBF16, int V>
bool launch_rows(const RouteArgs& a, hipStream_t st) {
  const bool grouped = a.top_groups < a.G;
  const bool by_logit = !a.bias && (!grouped || a.group_top == 1);
  if (!rows_fit(a, V, grouped)) return false;
  const int quads = (a.N + 3) / 4;
  const dim3 grid(min((quads + kRouteWaves - 1) / kRouteWaves, kRouteGroups)), block(64 * kRouteWaves);
  // K = 8, the K of this library's large workloads, has its rounds unrolled
  // where scores are compared (131072 x 256: 69 us in a loop, 63 unrolled).
  // Other K, and comparisons by logits (65536 x 384: 30.6 us in a loop, 29.2
  // unrolled), share the loop: each K is six more kernels to a type.
#define MB_R(L, G)                                                                               \
  do {                                                                                           \
    if (a.K == 8 && V >= 8 && !L)                                                                \
      hipLaunchKernelGGL((k_route_rows<kBF16, V, L, G, V >= 8 && !L ? 8 : 0>), grid, block, 0,   \
                         st, a, quads);                                                          \
    else                                                                                         \
      hipLaunchKernelGGL((k_route_rows<kBF16, V, L, G, 0>), grid, block, 0, st, a, quads);       \
  } while (0)
  if (by_logit) {
    if (grouped) MB_R(true, true);
    else MB_R(true, false);
  } else {
    if (grouped) MB_R(false, true);
    else MB_R(false, false);
  }
#undef MB_R
  return true;
}

template <bool kBF16>
void launch_route_t(const RouteArgs& a, hipStream_t st) {
  const int need = (a.E + 15) / 16;
  const bool done = need <= 1    ? launch_rows<kBF16, 1>(a, st)
                    : need <= 4  ? launch_rows<kBF16, 4>(a, st)
                    : need <= 8  ? launch_rows<kBF16, 8>(a, st)
                    : need <= 16 ? launch_rows<kBF16, 16>(a, st)
                    : need <= 24 ? launch_rows<kBF16, 24>(a, st)
                    : need <= 32 ? launch_rows<kBF16, 32>(a, st)
                                 : false;
  if (done) return;
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
