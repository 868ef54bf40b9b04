// api.hip — libmoebal's C ABI: argument checks, workspace layout, launches.
// The operations and conventions are documented in include/moebal.h.
#include <string.h>

#include <mutex>

#include "mb_internal.h"

namespace mb {

Geometry geometry(const mb_dims& d) {
  Geometry g;
  g.S = d.n_tokens / d.n_ranks;
  g.Eh = d.n_experts / d.n_ranks;
  g.NS = g.Eh + d.slots_per_rank;
  g.nbps = (g.S + kTokensPerBlock - 1) / kTokensPerBlock;
  g.nblk = g.nbps * d.n_ranks;
  return g;
}

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t drift_state_bytes(const mb_dims& d) {
  const size_t PR = (size_t)d.n_ranks * d.slots_per_rank;
  return align256(sizeof(mb_drift_header) + sizeof(int64_t) * d.n_experts +
                  2 * sizeof(int32_t) * PR);
}

WsLayout ws_layout(const mb_dims& d, const Geometry& g) {
  WsLayout L;
  size_t off = 0;
  const size_t per_block = (size_t)g.nblk * d.n_experts * sizeof(int32_t);
  L.blockcnt = off;
  off = align256(off + per_block);
  L.blockoff = off;
  off = align256(off + per_block);
  L.blockflags = off;
  off = align256(off + (size_t)g.nblk * sizeof(int32_t) + sizeof(int32_t));
  L.brank = off;
  off = align256(off + (size_t)d.n_tokens * d.top_k);
  L.expert_total = off;
  off = align256(off + (size_t)d.n_experts * sizeof(int32_t));
  L.pair_tab = off;
  off = align256(off + (size_t)d.n_ranks * d.n_experts * sizeof(PairEntry));
  L.host_list = off;
  off = align256(off + (size_t)host_list_cap(d) * sizeof(HostEntry));
  L.host_range = off;
  off = align256(off + (size_t)d.n_experts * sizeof(int2));
  L.total = off;
  return L;
}

}  // namespace mb

using namespace mb;

static int validate(const mb_dims* d) {
  if (!d) return MB_ERR_INVALID_ARG;
  if (d->n_ranks < 1 || d->n_ranks > kMaxRanks) return MB_ERR_INVALID_ARG;
  if (d->n_tokens < 0 || d->n_tokens % d->n_ranks) return MB_ERR_INVALID_ARG;
  if (d->n_experts < 1 || d->n_experts > kMaxExperts || d->n_experts % d->n_ranks)
    return MB_ERR_INVALID_ARG;
  if (d->top_k < 1 || d->top_k > d->n_experts || d->top_k > kMaxTopK) return MB_ERR_INVALID_ARG;
  if (d->slots_per_rank < 0 || d->slots_per_rank > kMaxSlots) return MB_ERR_INVALID_ARG;
  if (d->hidden < 1 || d->cap < 1) return MB_ERR_INVALID_ARG;
  if ((int64_t)d->n_tokens * d->top_k > INT32_MAX) return MB_ERR_INVALID_ARG;
  if ((int64_t)d->n_ranks * d->cap > INT32_MAX) return MB_ERR_INVALID_ARG;
  const int64_t row_in = row_bytes(d->dtype_in, d->hidden);
  if (!row_in) return MB_ERR_INVALID_ARG;
  if (d->dtype_out != MB_F32 && d->dtype_out != MB_BF16) return MB_ERR_INVALID_ARG;
  if (row_in % 16 || (int64_t)d->hidden * elt_bytes(d->dtype_out) % 16)
    return MB_ERR_INVALID_ARG;
  if (row_in / 16 > INT32_MAX) return MB_ERR_INVALID_ARG;
  // dispatch runs one wave per 1 KiB part of every token row, the combines
  // one per 512 bytes of output row (at least as many as per 512 fp8
  // elements of an expert row, which the fp8 combine uses)
  if ((int64_t)d->n_tokens * ((row_in / 16 + 63) / 64) > INT32_MAX)
    return MB_ERR_INVALID_ARG;
  if ((int64_t)d->n_tokens * (((int64_t)d->hidden * elt_bytes(d->dtype_out) / 8 + 63) / 64) >
      INT32_MAX)
    return MB_ERR_INVALID_ARG;
  if (scaled_rows(d->dtype_in) && d->hidden % 128) return MB_ERR_INVALID_ARG;
  return MB_OK;
}

// pos may be NULL only when there are no pairs (N == 0).
static bool plan_ptrs_ok(const mb_dims* d, const mb_plan_bufs* o) {
  return o && o->counts && o->load_pre && o->load_post && o->slot_quota && o->cu_seqlens &&
         (o->pos || d->n_tokens == 0) && o->row_src && o->status;
}

static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Memory a call reads, or writes.
struct Span {
  const void* at;
  int64_t bytes;
  bool written;
};

// No span that is written overlaps another: workgroups run in any order, so
// one's output could be another's input.
static bool outputs_apart(std::initializer_list<Span> spans) {
  for (const Span* a = spans.begin(); a != spans.end(); ++a)
    for (const Span* b = a + 1; b != spans.end(); ++b) {
      if (!(a->written || b->written) || a->bytes <= 0 || b->bytes <= 0) continue;
      const uintptr_t p = (uintptr_t)a->at, q = (uintptr_t)b->at;
      if (p < q + (uint64_t)b->bytes && q < p + (uint64_t)a->bytes) return false;
    }
  return true;
}

extern "C" {

int mb_version(void) { return MB_VERSION; }

const char* mb_strerror(int code) {
  switch (code) {
    case MB_OK: return "ok";
    case MB_ERR_INVALID_ARG: return "invalid argument (sizes outside the limits or null pointer)";
    case MB_ERR_WORKSPACE: return "workspace smaller than mb_plan_workspace_bytes()";
    case MB_ERR_HIP: return "HIP runtime error";
    case MB_ST_BAD_ID: return "status: an expert id outside [0, E)";
    case MB_ST_DUP_ID: return "status: a token lists one expert twice";
    case MB_ST_UNBALANCED: return "status: placement stopped with a rank above its target";
    case MB_ST_CAPACITY: return "status: a rank needs more rows than cap";
    default: return "unknown code";
  }
}

size_t mb_plan_workspace_bytes(const mb_dims* dims) {
  if (validate(dims) != MB_OK) return 0;
  const Geometry g = geometry(*dims);
  return ws_layout(*dims, g).total;
}

static int plan_impl(const mb_dims* dims, const int32_t* ids_dev, const int32_t* rank_speed,
                     const mb_drift_params* drift, void* drift_state, int repair, void* ws_dev,
                     size_t ws_bytes, const mb_plan_bufs* out, hipStream_t stream) {
  int rc = validate(dims);
  if (rc != MB_OK) return rc;
  if (!plan_ptrs_ok(dims, out) || !ws_dev || (dims->n_tokens > 0 && !ids_dev) ||
      (dims->slots_per_rank > 0 && !out->rep_expert) || !aligned16(ws_dev))
    return MB_ERR_INVALID_ARG;
  for (int r = 0; r < dims->n_ranks; ++r)
    if (rank_speed[r] < 1 || rank_speed[r] > MB_MAX_SPEED) return MB_ERR_INVALID_ARG;
  const Geometry g = geometry(*dims);
  const WsLayout L = ws_layout(*dims, g);
  if (ws_bytes < L.total) return MB_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(ws_dev);
  int32_t* blockcnt = reinterpret_cast<int32_t*>(ws + L.blockcnt);
  int32_t* blockoff = reinterpret_cast<int32_t*>(ws + L.blockoff);
  int32_t* blockflags = reinterpret_cast<int32_t*>(ws + L.blockflags);
  PairEntry* pair_tab = reinterpret_cast<PairEntry*>(ws + L.pair_tab);
  HostEntry* host_list = reinterpret_cast<HostEntry*>(ws + L.host_list);
  int2* host_range = reinterpret_cast<int2*>(ws + L.host_range);
  int32_t* expert_total = reinterpret_cast<int32_t*>(ws + L.expert_total);
  uint8_t* brank = ws + L.brank;

  // count -> per-source offsets and totals -> greedy placement -> lookup
  // tables -> per-pair rows, all on `stream`, no host synchronisation.
  // With one routing block per source rank, the block counts are d[s][e]
  // and every block offset is 0: k_count writes d itself, the scan is
  // skipped and k_plan sums c_e. With a few blocks per source and a small
  // table of block counts, the scan is skipped too: k_plan sums the table
  // into d[s][e] and c_e, and each k_assign block sums its source's earlier
  // blocks.
  const bool one_block = g.nbps == 1;
  const bool small = small_block_table(*dims, g);
  const bool scan = !one_block && !small;
  const bool tables_in_plan = dims->n_experts <= kPlanTableExperts;
  if (launch_count(*dims, g, ids_dev, one_block ? out->counts : blockcnt, blockflags, brank,
                   stream) != hipSuccess)
    return MB_ERR_HIP;
  if (scan &&
      launch_scan(*dims, g, blockcnt, blockoff, out->counts, expert_total, stream) != hipSuccess)
    return MB_ERR_HIP;
  if (launch_plan(*dims, g, *out, rank_speed, drift, drift_state, repair, blockflags,
                  scan ? expert_total : nullptr, small ? blockcnt : nullptr,
                  tables_in_plan ? pair_tab : nullptr, tables_in_plan ? host_list : nullptr,
                  tables_in_plan ? host_range : nullptr, stream) != hipSuccess)
    return MB_ERR_HIP;
  if (!tables_in_plan &&
      launch_tables(*dims, g, *out, pair_tab, host_list, host_range, stream) != hipSuccess)
    return MB_ERR_HIP;
  if (launch_assign(*dims, g, ids_dev, brank, scan ? blockoff : nullptr,
                    small ? blockcnt : nullptr, pair_tab, host_list, host_range, *out,
                    stream) != hipSuccess)
    return MB_ERR_HIP;
  return MB_OK;
}

int mb_plan(const mb_dims* dims, const int32_t* ids_dev, void* ws_dev, size_t ws_bytes,
            const mb_plan_bufs* out, hipStream_t stream) {
  // Equal speeds: every target is the water level T = ceil(N*K / P)
  // (ISER-MoE, HALO-Q Objective 1).
  int32_t ones[kMaxRanks];
  for (int r = 0; r < kMaxRanks; ++r) ones[r] = 1;
  return plan_impl(dims, ids_dev, ones, nullptr, nullptr, 0, ws_dev, ws_bytes, out, stream);
}

// ---- mb_plan_noalloc: mb_plan on a workspace the library holds ----------
//
// Every GPU the library runs on holds its own copy of `scratch`, at its own
// address, until the process ends. In host code the array's name is only a
// host-side stand-in: the device address comes from hipGetSymbolAddress,
// taken once per device with that device current, and only that address is
// handed to kernels.
static __device__ __align__(256) uint8_t scratch[MB_NOALLOC_WS_BYTES];

static constexpr int kMaxDevices = 64;
static std::mutex g_scratch_mu;
static void* g_scratch[kMaxDevices];

// Device address of `scratch` on the GPU that `stream` belongs to.
static int scratch_for(hipStream_t stream, void** out) {
  int dev = 0;
  if (hipStreamGetDevice(stream, &dev) != hipSuccess) return MB_ERR_HIP;
  if (dev < 0 || dev >= kMaxDevices) return MB_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch[dev]) {
    int cur = 0;
    if (hipGetDevice(&cur) != hipSuccess) return MB_ERR_HIP;
    if (cur != dev && hipSetDevice(dev) != hipSuccess) return MB_ERR_HIP;
    void* p = nullptr;
    const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (cur != dev && hipSetDevice(cur) != hipSuccess) return MB_ERR_HIP;
    if (e != hipSuccess || !p) return MB_ERR_HIP;
    g_scratch[dev] = p;
  }
  *out = g_scratch[dev];
  return MB_OK;
}

int mb_plan_noalloc(const mb_dims* dims, const int32_t* ids_dev, const mb_plan_bufs* out,
                    hipStream_t stream) {
  const int rc = validate(dims);
  if (rc != MB_OK) return rc;
  const size_t need = ws_layout(*dims, geometry(*dims)).total;
  if (need > MB_NOALLOC_WS_BYTES) return MB_ERR_WORKSPACE;
  void* ws = nullptr;
  const int src = scratch_for(stream, &ws);
  if (src != MB_OK) return src;
  int32_t ones[kMaxRanks];
  for (int r = 0; r < kMaxRanks; ++r) ones[r] = 1;
  return plan_impl(dims, ids_dev, ones, nullptr, nullptr, 0, ws, MB_NOALLOC_WS_BYTES, out,
                   stream);
}

int mb_plan_weighted(const mb_dims* dims, const int32_t* ids_dev, const int32_t* rank_speed,
                     void* ws_dev, size_t ws_bytes, const mb_plan_bufs* out,
                     hipStream_t stream) {
  if (!rank_speed) return MB_ERR_INVALID_ARG;
  return plan_impl(dims, ids_dev, rank_speed, nullptr, nullptr, 0, ws_dev, ws_bytes, out,
                   stream);
}

size_t mb_drift_state_bytes(const mb_dims* dims) {
  if (validate(dims) != MB_OK) return 0;
  return drift_state_bytes(*dims);
}

int mb_plan_ex(const mb_dims* dims, const int32_t* ids_dev, const mb_plan_options* opt,
               void* ws_dev, size_t ws_bytes, const mb_plan_bufs* out, hipStream_t stream) {
  if (!opt) return MB_ERR_INVALID_ARG;
  const mb_drift_params* prm = opt->drift;
  if ((prm != nullptr) != (opt->drift_state != nullptr)) return MB_ERR_INVALID_ARG;
  if (prm) {
    if (!aligned16(opt->drift_state)) return MB_ERR_INVALID_ARG;
    if (prm->delta_den < 1 || prm->delta_num < 0 || prm->delta_num > prm->delta_den ||
        prm->window < 1 || prm->window > MB_MAX_WINDOW || prm->check_every < 1 ||
        prm->tol_num < 0 || prm->tol_den < 0)
      return MB_ERR_INVALID_ARG;
  }
  int32_t ones[kMaxRanks];
  for (int r = 0; r < kMaxRanks; ++r) ones[r] = 1;
  return plan_impl(dims, ids_dev, opt->rank_speed ? opt->rank_speed : ones, prm,
                   opt->drift_state, opt->quota_repair != 0, ws_dev, ws_bytes, out, stream);
}

int mb_plan_drift(const mb_dims* dims, const int32_t* ids_dev, const int32_t* rank_speed,
                  const mb_drift_params* params, void* state_dev, void* ws_dev,
                  size_t ws_bytes, const mb_plan_bufs* out, hipStream_t stream) {
  if (!params || !state_dev) return MB_ERR_INVALID_ARG;
  const mb_plan_options opt = {rank_speed, params, state_dev, 0};
  return mb_plan_ex(dims, ids_dev, &opt, ws_dev, ws_bytes, out, stream);
}

int mb_dispatch(const mb_dims* dims, const mb_plan_bufs* plan, const void* x_dev,
                const float* x_scale_dev, void* buf_dev, float* buf_scale_dev,
                hipStream_t stream) {
  int rc = validate(dims);
  if (rc != MB_OK) return rc;
  if (!plan || (dims->n_tokens > 0 && (!plan->pos || !x_dev)) || !plan->status || !buf_dev)
    return MB_ERR_INVALID_ARG;
  if (!aligned16(x_dev) || !aligned16(buf_dev)) return MB_ERR_INVALID_ARG;
  if (scaled_rows(dims->dtype_in) && (!x_scale_dev || !buf_scale_dev)) return MB_ERR_INVALID_ARG;
  if (dims->dtype_in == MB_MX4 && (!aligned4(x_scale_dev) || !aligned4(buf_scale_dev)))
    return MB_ERR_INVALID_ARG;
  return launch_dispatch(*dims, *plan, x_dev, x_scale_dev, buf_dev, buf_scale_dev, stream) ==
                 hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

int mb_combine(const mb_dims* dims, const mb_plan_bufs* plan, const void* y_exp_dev,
               const float* w_dev, void* y_dev, hipStream_t stream) {
  int rc = validate(dims);
  if (rc != MB_OK) return rc;
  if (!plan || !plan->status || !y_exp_dev ||
      (dims->n_tokens > 0 && (!plan->pos || !w_dev || !y_dev)))
    return MB_ERR_INVALID_ARG;
  if (!aligned16(y_exp_dev) || !aligned16(y_dev)) return MB_ERR_INVALID_ARG;
  return launch_combine(*dims, *plan, y_exp_dev, w_dev, y_dev, stream) == hipSuccess ? MB_OK
                                                                                     : MB_ERR_HIP;
}

int mb_combine_fp8(const mb_dims* dims, const mb_plan_bufs* plan, const uint8_t* y_exp_dev,
                   const float* y_scale_dev, const float* w_dev, void* y_dev,
                   hipStream_t stream) {
  int rc = validate(dims);
  if (rc != MB_OK) return rc;
  if (dims->hidden % 128) return MB_ERR_INVALID_ARG;
  if (!plan || !plan->status || !y_exp_dev || !y_scale_dev ||
      (dims->n_tokens > 0 && (!plan->pos || !w_dev || !y_dev)))
    return MB_ERR_INVALID_ARG;
  if (!aligned16(y_exp_dev) || !aligned16(y_dev) || ((uintptr_t)y_scale_dev & 3u))
    return MB_ERR_INVALID_ARG;
  return launch_combine_fp8(*dims, *plan, y_exp_dev, y_scale_dev, w_dev, y_dev, stream) ==
                 hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

int mb_route(const mb_route_params* prm, const void* logits_dev, const float* bias_dev,
             int32_t* ids_dev, float* w_dev, hipStream_t stream) {
  if (!prm) return MB_ERR_INVALID_ARG;
  const mb_route_params& p = *prm;
  if (p.n_tokens < 0 || p.n_experts < 1 || p.n_experts > kMaxExperts) return MB_ERR_INVALID_ARG;
  if (p.n_groups < 1 || p.n_groups > kMaxGroups || p.n_experts % p.n_groups)
    return MB_ERR_INVALID_ARG;
  const int size = p.n_experts / p.n_groups;
  if (p.top_groups < 1 || p.top_groups > p.n_groups) return MB_ERR_INVALID_ARG;
  if (p.group_top < 1 || p.group_top > 2 || p.group_top > size) return MB_ERR_INVALID_ARG;
  if (p.top_k < 1 || p.top_k > kMaxTopK || p.top_k > p.top_groups * size)
    return MB_ERR_INVALID_ARG;
  if (p.dtype != MB_F32 && p.dtype != MB_BF16) return MB_ERR_INVALID_ARG;
  if (p.score != MB_SCORE_SOFTMAX && p.score != MB_SCORE_SIGMOID) return MB_ERR_INVALID_ARG;
  if (!(p.scale - p.scale == 0.0f)) return MB_ERR_INVALID_ARG;  // NaN or infinite
  if (p.n_tokens > kMaxWaves) return MB_ERR_INVALID_ARG;
  if (p.n_tokens > 0 && (!logits_dev || !ids_dev || !w_dev)) return MB_ERR_INVALID_ARG;
  if (!aligned16(logits_dev) || !aligned4(bias_dev) || !aligned4(ids_dev) || !aligned4(w_dev))
    return MB_ERR_INVALID_ARG;
  const int64_t n = p.n_tokens, picks = n * p.top_k * 4;
  if (!outputs_apart({{logits_dev, n * p.n_experts * elt_bytes(p.dtype), false},
                      {bias_dev, n && bias_dev ? (int64_t)p.n_experts * 4 : 0, false},
                      {ids_dev, picks, true},
                      {w_dev, picks, true}}))
    return MB_ERR_INVALID_ARG;
  return launch_route(p, logits_dev, bias_dev, ids_dev, w_dev, stream) == hipSuccess ? MB_OK
                                                                                     : MB_ERR_HIP;
}

int mb_rmsnorm_fp8(int32_t n_rows, int32_t hidden, int32_t dtype, float eps, const void* x_dev,
                   const void* residual_dev, const void* weight_dev, void* residual_out_dev,
                   void* y_dev, uint8_t* q_dev, float* q_scale_dev, hipStream_t stream) {
  if (n_rows < 0 || n_rows > kMaxWaves / 4 || hidden < 128 || hidden % 128 ||
      hidden > MB_MAX_NORM_HIDDEN)
    return MB_ERR_INVALID_ARG;
  if (dtype != MB_F32 && dtype != MB_BF16) return MB_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(eps - eps == 0.0f)) return MB_ERR_INVALID_ARG;
  if (residual_out_dev && !residual_dev) return MB_ERR_INVALID_ARG;
  if (n_rows > 0 && (!x_dev || !weight_dev || !q_dev || !q_scale_dev)) return MB_ERR_INVALID_ARG;
  if (!aligned16(x_dev) || !aligned16(residual_dev) || !aligned16(weight_dev) ||
      !aligned16(residual_out_dev) || !aligned16(y_dev) || !aligned16(q_dev) ||
      !aligned4(q_scale_dev))
    return MB_ERR_INVALID_ARG;
  // in place, the input's span is the written one
  const int64_t elems = (int64_t)n_rows * hidden, rows = elems * elt_bytes(dtype);
  const bool over_x = residual_out_dev && residual_out_dev == x_dev;
  const bool over_res = residual_out_dev && residual_out_dev == residual_dev;
  if (!outputs_apart({{x_dev, rows, over_x},
                      {residual_dev, residual_dev && !(over_x && over_res) ? rows : 0, over_res},
                      {residual_out_dev, residual_out_dev && !over_x && !over_res ? rows : 0, true},
                      {weight_dev, n_rows ? hidden * elt_bytes(dtype) : 0, false},
                      {y_dev, y_dev ? rows : 0, true},
                      {q_dev, elems, true},
                      {q_scale_dev, elems / 32, true}}))
    return MB_ERR_INVALID_ARG;
  return launch_rmsnorm_fp8(n_rows, hidden, dtype == MB_BF16, eps, x_dev, residual_dev, weight_dev,
                            residual_out_dev, y_dev, q_dev, q_scale_dev, stream) == hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

// Sizes shared by the two directions of the 4-bit rows.
static bool mx4_rows_ok(int32_t n_rows, int32_t hidden, int32_t dtype) {
  if (n_rows < 0 || hidden < 32 || hidden % 32) return false;
  if (dtype != MB_F32 && dtype != MB_BF16) return false;
  // a wave per 512 elements of a row, in launches of fewer than 2^32 threads
  return (int64_t)n_rows * ((hidden + 511) / 512) <= kMaxWaves;
}

int mb_quantize_mx4(int32_t n_rows, int32_t hidden, int32_t dtype, int32_t act, const void* x_dev,
                    const int32_t* row_src_dev, uint8_t* q_dev, uint8_t* q_scale_dev,
                    hipStream_t stream) {
  if (!mx4_rows_ok(n_rows, hidden, dtype)) return MB_ERR_INVALID_ARG;
  if (act != MB_ACT_NONE && act != MB_ACT_SWIGLU) return MB_ERR_INVALID_ARG;
  if (n_rows > 0 && (!x_dev || !q_dev || !q_scale_dev)) return MB_ERR_INVALID_ARG;
  if (!aligned16(x_dev) || !aligned16(q_dev) || !aligned4(row_src_dev)) return MB_ERR_INVALID_ARG;
  const int64_t elems = (int64_t)n_rows * hidden;
  if (!outputs_apart({{x_dev, elems * elt_bytes(dtype) * (act == MB_ACT_SWIGLU ? 2 : 1), false},
                      {row_src_dev, row_src_dev ? (int64_t)n_rows * 4 : 0, false},
                      {q_dev, elems / 2, true},
                      {q_scale_dev, elems / 32, true}}))
    return MB_ERR_INVALID_ARG;
  return launch_quantize_mx4(n_rows, hidden, dtype == MB_BF16, act == MB_ACT_SWIGLU, x_dev,
                             row_src_dev, q_dev, q_scale_dev, stream) == hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

int mb_dequantize_mx4(int32_t n_rows, int32_t hidden, int32_t dtype, const uint8_t* q_dev,
                      const uint8_t* q_scale_dev, void* x_dev, hipStream_t stream) {
  if (!mx4_rows_ok(n_rows, hidden, dtype)) return MB_ERR_INVALID_ARG;
  if (n_rows > 0 && (!x_dev || !q_dev || !q_scale_dev)) return MB_ERR_INVALID_ARG;
  if (!aligned16(x_dev) || !aligned16(q_dev)) return MB_ERR_INVALID_ARG;
  const int64_t elems = (int64_t)n_rows * hidden;
  if (!outputs_apart({{q_dev, elems / 2, false},
                      {q_scale_dev, elems / 32, false},
                      {x_dev, elems * elt_bytes(dtype), true}}))
    return MB_ERR_INVALID_ARG;
  return launch_dequantize_mx4(n_rows, hidden, dtype == MB_BF16, q_dev, q_scale_dev, x_dev,
                               stream) == hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

int mb_expert_mx4(const mb_dims* dims, const mb_plan_bufs* plan, int32_t n_out, int32_t k_in,
                  const uint8_t* a_dev, const uint8_t* a_scale_dev, const uint8_t* w_dev,
                  const uint8_t* w_scale_dev, void* y_dev, hipStream_t stream) {
  const int rc = validate(dims);
  if (rc != MB_OK) return rc;
  if (n_out < 1 || n_out > kMaxExpertDim || n_out * elt_bytes(dims->dtype_out) % 16)
    return MB_ERR_INVALID_ARG;
  if (k_in < 128 || k_in > kMaxExpertDim || k_in % 128) return MB_ERR_INVALID_ARG;
  if (!plan || !plan->status || !plan->cu_seqlens ||
      (dims->slots_per_rank > 0 && !plan->rep_expert) || !a_dev || !a_scale_dev || !w_dev ||
      !w_scale_dev || !y_dev)
    return MB_ERR_INVALID_ARG;
  if (!aligned16(a_dev) || !aligned16(w_dev) || !aligned16(y_dev) || !aligned4(a_scale_dev) ||
      !aligned4(w_scale_dev))
    return MB_ERR_INVALID_ARG;
  // a tile's rows are numbered in int32, also those behind the last region's end
  if ((int64_t)dims->n_ranks * dims->cap > INT32_MAX - (kMaxTileRows - 1))
    return MB_ERR_INVALID_ARG;
  const Geometry g = geometry(*dims);
  // output tiles of at least 16 rows x 16 columns are numbered in int32
  const int64_t row_tiles = (int64_t)dims->n_ranks * dims->cap / 16 + (int64_t)dims->n_ranks * g.NS;
  if (row_tiles * ((n_out + 15) / 16) > INT32_MAX) return MB_ERR_INVALID_ARG;
  const int64_t rows = dims->n_tokens ? (int64_t)dims->n_ranks * dims->cap : 0;
  const int64_t weights = (int64_t)dims->n_experts * n_out;
  if (!outputs_apart({{y_dev, rows * n_out * elt_bytes(dims->dtype_out), true},
                      {a_dev, rows * k_in / 2, false},
                      {a_scale_dev, rows * k_in / 32, false},
                      {w_dev, weights * k_in / 2, false},
                      {w_scale_dev, weights * k_in / 32, false},
                      {plan->cu_seqlens, (int64_t)dims->n_ranks * (g.NS + 1) * 4, false},
                      {plan->rep_expert, (int64_t)dims->n_ranks * dims->slots_per_rank * 4, false},
                      {plan->status, 16, false}}))
    return MB_ERR_INVALID_ARG;
  return launch_expert_mx4(*dims, g, *plan, n_out, k_in, a_dev, a_scale_dev, w_dev, w_scale_dev,
                           y_dev, stream) == hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

// What the products of bf16 rows share: the sizes, the plan and the region's
// rows. `rows` and `weights`: rows of the dispatch layout, and of all experts.
static bool bf16_product_ok(const mb_dims* dims, const mb_plan_bufs* plan, int32_t n_out,
                            int32_t k_in, int64_t* rows, int64_t* weights) {
  if (validate(dims) != MB_OK) return false;
  if (n_out < 8 || n_out > kMaxExpertDim || n_out % 8) return false;
  if (k_in < 8 || k_in > kMaxExpertDim || k_in % 8) return false;
  if (!plan || !plan->status || !plan->cu_seqlens ||
      (dims->slots_per_rank > 0 && !plan->rep_expert))
    return false;
  // a tile's rows are numbered in int32, also those behind the last region's end
  if ((int64_t)dims->n_ranks * dims->cap > INT32_MAX - (kMaxTileRows - 1)) return false;
  const Geometry g = geometry(*dims);
  // output tiles of at least 16 rows x 16 columns, of the rows and of the
  // weights, are numbered in int32
  const int64_t row_tiles = (int64_t)dims->n_ranks * dims->cap / 16 + (int64_t)dims->n_ranks * g.NS;
  const int64_t wide = ((n_out > k_in ? n_out : k_in) + 15) / 16;
  if (row_tiles * wide > INT32_MAX) return false;
  if ((int64_t)dims->n_experts * ((n_out + 127) / 128) * ((k_in + 127) / 128) > INT32_MAX)
    return false;
  *rows = dims->n_tokens ? (int64_t)dims->n_ranks * dims->cap : 0;
  *weights = (int64_t)dims->n_experts * n_out;
  return true;
}

// Nothing written overlaps the plan's arrays that the products read.
static bool apart_from_plan(const mb_dims* dims, const mb_plan_bufs* plan, Span written) {
  const Geometry g = geometry(*dims);
  written.written = true;
  return outputs_apart(
      {written,
       {plan->cu_seqlens, (int64_t)dims->n_ranks * (g.NS + 1) * 4, false},
       {plan->rep_expert, (int64_t)dims->n_ranks * dims->slots_per_rank * 4, false},
       {plan->status, 16, false}});
}

int mb_expert_bf16(const mb_dims* dims, const mb_plan_bufs* plan, int32_t act, int32_t n_out,
                   int32_t k_in, const uint16_t* a_dev, const uint16_t* w_dev, void* y_dev,
                   uint16_t* pre_dev, hipStream_t stream) {
  int64_t rows, weights;
  if (!bf16_product_ok(dims, plan, n_out, k_in, &rows, &weights)) return MB_ERR_INVALID_ARG;
  if (act != MB_ACT_NONE && act != MB_ACT_SWIGLU) return MB_ERR_INVALID_ARG;
  const bool gated = act == MB_ACT_SWIGLU;
  if (!a_dev || !w_dev || !y_dev || (pre_dev && !gated)) return MB_ERR_INVALID_ARG;
  if (!aligned16(a_dev) || !aligned16(w_dev) || !aligned16(y_dev) || !aligned16(pre_dev))
    return MB_ERR_INVALID_ARG;
  const Span y = {y_dev, rows * n_out * (gated ? 2 : elt_bytes(dims->dtype_out)), true};
  const Span pre = {pre_dev, pre_dev ? rows * n_out * 4 : 0, true};
  if (!outputs_apart({y, pre, {a_dev, rows * k_in * 2, false},
                      {w_dev, weights * k_in * (gated ? 4 : 2), false}}) ||
      !apart_from_plan(dims, plan, y) || !apart_from_plan(dims, plan, pre))
    return MB_ERR_INVALID_ARG;
  return launch_expert_bf16(*dims, geometry(*dims), *plan, gated, n_out, k_in, a_dev, w_dev, y_dev,
                            pre_dev, stream) == hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

int mb_expert_bf16_dgrad(const mb_dims* dims, const mb_plan_bufs* plan, int32_t act, int32_t n_out,
                         int32_t k_in, const uint16_t* dy_dev, const uint16_t* w_dev,
                         const uint16_t* pre_dev, void* da_dev, hipStream_t stream) {
  int64_t rows, weights;
  if (!bf16_product_ok(dims, plan, n_out, k_in, &rows, &weights)) return MB_ERR_INVALID_ARG;
  if (act != MB_ACT_NONE && act != MB_ACT_SWIGLU) return MB_ERR_INVALID_ARG;
  const bool gated = act == MB_ACT_SWIGLU;
  if (!dy_dev || !w_dev || !da_dev || (pre_dev != nullptr) != gated) return MB_ERR_INVALID_ARG;
  if (!aligned16(dy_dev) || !aligned16(w_dev) || !aligned16(da_dev) || !aligned16(pre_dev))
    return MB_ERR_INVALID_ARG;
  const Span da = {da_dev, rows * k_in * (gated ? 4 : elt_bytes(dims->dtype_out)), true};
  if (!outputs_apart({da, {dy_dev, rows * n_out * 2, false}, {w_dev, weights * k_in * 2, false},
                      {pre_dev, pre_dev ? rows * k_in * 4 : 0, false}}) ||
      !apart_from_plan(dims, plan, da))
    return MB_ERR_INVALID_ARG;
  return launch_expert_bf16_dgrad(*dims, geometry(*dims), *plan, gated, n_out, k_in, dy_dev, w_dev,
                                  pre_dev, da_dev, stream) == hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

int mb_expert_bf16_wgrad(const mb_dims* dims, const mb_plan_bufs* plan, int32_t n_out, int32_t k_in,
                         int32_t dtype, int32_t accumulate, const uint16_t* dy_dev,
                         const uint16_t* a_dev, void* dw_dev, hipStream_t stream) {
  int64_t rows, weights;
  if (!bf16_product_ok(dims, plan, n_out, k_in, &rows, &weights)) return MB_ERR_INVALID_ARG;
  if (dtype != MB_F32 && dtype != MB_BF16) return MB_ERR_INVALID_ARG;
  if (!dw_dev || (dims->n_tokens > 0 && (!dy_dev || !a_dev))) return MB_ERR_INVALID_ARG;
  if (!aligned16(dy_dev) || !aligned16(a_dev) || !aligned16(dw_dev)) return MB_ERR_INVALID_ARG;
  const Span dw = {dw_dev, weights * k_in * elt_bytes(dtype), true};
  if (!outputs_apart({dw, {dy_dev, rows * n_out * 2, false}, {a_dev, rows * k_in * 2, false}}) ||
      !apart_from_plan(dims, plan, dw))
    return MB_ERR_INVALID_ARG;
  return launch_expert_bf16_wgrad(*dims, geometry(*dims), *plan, n_out, k_in, accumulate != 0,
                                  dtype == MB_BF16, dy_dev, a_dev, dw_dev, stream) == hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

int mb_combine_grad(const mb_dims* dims, const mb_plan_bufs* plan, const void* dy_dev,
                    const void* y_exp_dev, const float* w_dev, void* dy_exp_dev, float* dw_dev,
                    hipStream_t stream) {
  const int rc = validate(dims);
  if (rc != MB_OK) return rc;
  if (!plan || !plan->status || (!dy_exp_dev && !dw_dev)) return MB_ERR_INVALID_ARG;
  if (dims->n_tokens > 0 && (!plan->pos || !dy_dev || (dw_dev && !y_exp_dev) ||
                             (dy_exp_dev && !w_dev)))
    return MB_ERR_INVALID_ARG;
  if (!aligned16(dy_dev) || !aligned16(y_exp_dev) || !aligned16(dy_exp_dev) || !aligned4(w_dev) ||
      !aligned4(dw_dev))
    return MB_ERR_INVALID_ARG;
  const int64_t row = dims->hidden * elt_bytes(dims->dtype_out), pairs = (int64_t)dims->n_tokens * dims->top_k;
  const int64_t rows = dims->n_tokens ? (int64_t)dims->n_ranks * dims->cap : 0;
  if (!outputs_apart({{dy_exp_dev, dy_exp_dev ? rows * row : 0, true},
                      {dw_dev, dw_dev ? pairs * 4 : 0, true},
                      {dy_dev, dims->n_tokens * row, false},
                      {y_exp_dev, dw_dev ? rows * row : 0, false},
                      {w_dev, dy_exp_dev ? pairs * 4 : 0, false},
                      {plan->pos, pairs * 4, false},
                      {plan->status, 16, false}}))
    return MB_ERR_INVALID_ARG;
  return launch_combine_grad(*dims, *plan, dy_dev, y_exp_dev, w_dev, dy_exp_dev, dw_dev, stream) ==
                 hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

static bool lora_ok(const mb_lora_params* p) {
  if (!p || p->n_rows < 0 || p->n_rows > kMaxLoraRows) return false;
  if (p->n_out < 8 || p->n_out > kMaxExpertDim || p->n_out % 8) return false;
  if (p->k_in < 8 || p->k_in > kMaxExpertDim || p->k_in % 8) return false;
  if (p->rank < 8 || p->rank > MB_MAX_LORA_RANK || p->rank % 8) return false;
  if (p->n_adapters < 1 || p->n_adapters > kMaxAdapters) return false;
  if (p->dtype_out != MB_F32 && p->dtype_out != MB_BF16) return false;
  // output tiles of at least 16 x 16 are numbered in int32
  return ((int64_t)p->n_rows + 15) / 16 * ((p->n_out + 15) / 16) <= INT32_MAX;
}

size_t mb_lora_workspace_bytes(const mb_lora_params* prm) {
  if (!lora_ok(prm)) return 0;
  const size_t bytes = lora_workspace_floats(*prm) * sizeof(float);
  return align256(bytes ? bytes : 1);
}

int mb_project_lora(const mb_lora_params* prm, const uint16_t* x_dev, const uint16_t* w_dev,
                    const uint16_t* lora_a_dev, const uint16_t* lora_b_dev,
                    const float* scale_dev, const int32_t* adapter_dev, void* ws_dev,
                    size_t ws_bytes, void* y_dev, hipStream_t stream) {
  if (!lora_ok(prm)) return MB_ERR_INVALID_ARG;
  const mb_lora_params& p = *prm;
  if (p.n_rows > 0 && (!x_dev || !w_dev || !lora_a_dev || !lora_b_dev || !scale_dev ||
                       !adapter_dev || !ws_dev || !y_dev))
    return MB_ERR_INVALID_ARG;
  if (!aligned16(x_dev) || !aligned16(w_dev) || !aligned16(lora_a_dev) || !aligned16(lora_b_dev) ||
      !aligned4(scale_dev) || !aligned4(adapter_dev) || !aligned16(ws_dev) || !aligned16(y_dev))
    return MB_ERR_INVALID_ARG;
  const size_t need = mb_lora_workspace_bytes(prm);
  if (p.n_rows > 0 && ws_bytes < need) return MB_ERR_WORKSPACE;
  const int64_t any = p.n_rows > 0, n = p.n_out, k = p.k_in, low = (int64_t)p.n_adapters * p.rank;
  if (!outputs_apart({{y_dev, p.n_rows * n * elt_bytes(p.dtype_out), true},
                      {ws_dev, any * (int64_t)need, true},
                      {x_dev, p.n_rows * k * 2, false},
                      {w_dev, any * n * k * 2, false},
                      {lora_a_dev, any * low * k * 2, false},
                      {lora_b_dev, any * low * n * 2, false},
                      {scale_dev, any * p.n_adapters * 4, false},
                      {adapter_dev, (int64_t)p.n_rows * 4, false}}))
    return MB_ERR_INVALID_ARG;
  return launch_project_lora(p, x_dev, w_dev, lora_a_dev, lora_b_dev, scale_dev, adapter_dev,
                             static_cast<float*>(ws_dev), y_dev, stream) == hipSuccess
             ? MB_OK
             : MB_ERR_HIP;
}

int mb_plan_status(const mb_plan_bufs* plan, hipStream_t stream, int32_t host_status[4]) {
  if (!plan || !plan->status || !host_status) return MB_ERR_INVALID_ARG;
  if (hipMemcpyAsync(host_status, plan->status, 4 * sizeof(int32_t), hipMemcpyDeviceToHost,
                     stream) != hipSuccess)
    return MB_ERR_HIP;
  if (hipStreamSynchronize(stream) != hipSuccess) return MB_ERR_HIP;
  return MB_OK;
}

}  // extern "C"
