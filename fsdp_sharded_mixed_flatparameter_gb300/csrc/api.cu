// api.cu -- the C-ABI entry points of libzeroshard (declared in
// include/zero_shard.h): argument checking, per-step scalars, dispatch to the
// kernel launchers, and the per-thread error message.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "adam_scalars.cuh"
#include "common.cuh"
#include "kernels.h"
#include "rounding.cuh"

namespace zs {

static thread_local char g_msg[512] = "";

zero_status fail(zero_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return st;
}

zero_status check_launch(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(ZERO_ECUDA, "%s: %s", what, cudaGetErrorString(e));
  return ZERO_OK;
}

static bool valid_dtype(int d) { return d == ZERO_F32 || d == ZERO_BF16 || d == ZERO_F16; }

}  // namespace zs

using zs::fail;

extern "C" {

const char* zero_status_string(zero_status s) {
  switch (s) {
    case ZERO_OK: return "ZERO_OK";
    case ZERO_EINVAL: return "ZERO_EINVAL: invalid argument";
    case ZERO_ECUDA: return "ZERO_ECUDA: CUDA runtime error";
  }
  return "unknown zero_status";
}

const char* zero_last_error(void) { return zs::g_msg; }

zero_status zero_shard_range(int64_t total, int32_t world_size, int32_t rank, int64_t* start, int64_t* end) {
  if (start == nullptr || end == nullptr) return fail(ZERO_EINVAL, "zero_shard_range: NULL output");
  if (total < 0) return fail(ZERO_EINVAL, "zero_shard_range: total %lld < 0", (long long)total);
  if (world_size < 1) return fail(ZERO_EINVAL, "zero_shard_range: world_size %d < 1", world_size);
  if (rank < 0 || rank >= world_size)
    return fail(ZERO_EINVAL, "zero_shard_range: rank %d not in [0, %d)", rank, world_size);
  // chunk = ceil(total / world) without overflow for totals near INT64_MAX
  const int64_t chunk = total / world_size + (total % world_size != 0 ? 1 : 0);
  const int64_t s = (chunk != 0 && rank > (total / chunk)) ? total : static_cast<int64_t>(rank) * chunk;
  const int64_t lo = s < total ? s : total;
  const int64_t hi = (chunk > total - lo) ? total : lo + chunk;
  *start = lo;
  *end = hi;
  return ZERO_OK;
}

zero_status zero_tensor_table(const void* const* ptrs, const int64_t* numels, int32_t n_tensors,
                              zero_tensor* table, int64_t* total) {
  if (n_tensors < 0) return fail(ZERO_EINVAL, "zero_tensor_table: n_tensors %d < 0", n_tensors);
  if (total == nullptr) return fail(ZERO_EINVAL, "zero_tensor_table: NULL total");
  if (n_tensors > 0 && (numels == nullptr || table == nullptr))
    return fail(ZERO_EINVAL, "zero_tensor_table: NULL numels or table");
  int64_t acc = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (numels[i] < 0) return fail(ZERO_EINVAL, "zero_tensor_table: numel[%d] = %lld < 0", i, (long long)numels[i]);
    if (numels[i] > INT64_MAX - acc) return fail(ZERO_EINVAL, "zero_tensor_table: total overflows int64");
    acc += numels[i];
  }
  int64_t off = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    table[i].ptr = ptrs ? ptrs[i] : nullptr;
    table[i].numel = numels[i];
    table[i].flat_offset = off;
    off += numels[i];
  }
  *total = acc;
  return ZERO_OK;
}

// Optional fused-norm workspace of the flatten / accumulate calls: NULL, or
// room for one binary64 partial per 32768 output elements, 8-byte aligned.
static zero_status check_norm_ws(const char* who, const void* ws, size_t ws_bytes, int64_t n) {
  if (ws == nullptr) return ZERO_OK;
  const size_t need = zero_grad_sqnorm_workspace_bytes(n);
  if (ws_bytes < need) return fail(ZERO_EINVAL, "%s: norm workspace %zu bytes < %zu needed", who, ws_bytes, need);
  if (!zs::aligned(ws, 8)) return fail(ZERO_EINVAL, "%s: norm workspace not 8-byte aligned", who);
  return ZERO_OK;
}

zero_status zero_flatten_cast(const zero_tensor* d_table, int32_t n_tensors, int64_t total, zero_dtype src_dtype,
                              int64_t shard_start, int64_t shard_end, float scale, const float* d_scale,
                              int32_t accumulate, float* d_dst, int32_t* d_found_nonfinite, void* d_norm_ws,
                              size_t norm_ws_bytes, void* stream) {
  if (n_tensors < 0) return fail(ZERO_EINVAL, "zero_flatten_cast: n_tensors %d < 0", n_tensors);
  if (n_tensors > 0 && d_table == nullptr) return fail(ZERO_EINVAL, "zero_flatten_cast: NULL d_table");
  if (total < 0 || (n_tensors == 0 && total != 0))
    return fail(ZERO_EINVAL, "zero_flatten_cast: total %lld does not fit %d tensors", (long long)total, n_tensors);
  if (shard_start < 0 || shard_start > shard_end || shard_end > total)
    return fail(ZERO_EINVAL, "zero_flatten_cast: shard [%lld, %lld) outside [0, %lld]", (long long)shard_start,
                (long long)shard_end, (long long)total);
  if (!zs::valid_dtype(src_dtype)) return fail(ZERO_EINVAL, "zero_flatten_cast: bad src_dtype %d", (int)src_dtype);
  if (accumulate < 0 || accumulate > 2) return fail(ZERO_EINVAL, "zero_flatten_cast: accumulate must be 0, 1 or 2");
  if (!std::isfinite(scale)) return fail(ZERO_EINVAL, "zero_flatten_cast: non-finite scale");
  if (shard_end > shard_start && d_dst == nullptr && (d_norm_ws == nullptr || accumulate != 0))
    return fail(ZERO_EINVAL, "zero_flatten_cast: NULL d_dst needs a norm workspace and accumulate == 0");
  if (accumulate == 2 && shard_end > shard_start && d_norm_ws == nullptr)
    return fail(ZERO_EINVAL, "zero_flatten_cast: accumulate == 2 (norm of the sum only) needs a norm workspace");
  const zero_status w = check_norm_ws("zero_flatten_cast", d_norm_ws, norm_ws_bytes, shard_end - shard_start);
  if (w != ZERO_OK) return w;
  if (shard_end == shard_start) return ZERO_OK;
  return zs::launch_flatten(d_table, n_tensors, src_dtype, shard_start, shard_end, scale, d_scale, accumulate,
                            d_dst, d_found_nonfinite, static_cast<double*>(d_norm_ws), zs::as_stream(stream));
}

zero_status zero_accum(float* d_acc, const void* d_src, zero_dtype src_dtype, int64_t n, float scale,
                       const float* d_scale, int32_t accumulate, int32_t* d_found_nonfinite, void* d_norm_ws,
                       size_t norm_ws_bytes, void* stream) {
  if (n < 0) return fail(ZERO_EINVAL, "zero_accum: n %lld < 0", (long long)n);
  if (!zs::valid_dtype(src_dtype)) return fail(ZERO_EINVAL, "zero_accum: bad src_dtype %d", (int)src_dtype);
  if (accumulate != 0 && accumulate != 1) return fail(ZERO_EINVAL, "zero_accum: accumulate must be 0 or 1");
  if (!std::isfinite(scale)) return fail(ZERO_EINVAL, "zero_accum: non-finite scale");
  if (n > 0 && (d_acc == nullptr || d_src == nullptr)) return fail(ZERO_EINVAL, "zero_accum: NULL buffer");
  const zero_status w = check_norm_ws("zero_accum", d_norm_ws, norm_ws_bytes, n);
  if (w != ZERO_OK) return w;
  if (n == 0) return ZERO_OK;
  return zs::launch_accum(d_acc, d_src, src_dtype, n, scale, d_scale, accumulate, d_found_nonfinite,
                          static_cast<double*>(d_norm_ws), zs::as_stream(stream));
}

zero_status zero_reduce_chunks(float* d_acc, const void* d_chunks, zero_dtype src_dtype, int32_t n_chunks,
                               int64_t chunk_stride, int64_t n, float scale, const float* d_scale,
                               int32_t accumulate, int32_t* d_found_nonfinite, void* d_norm_ws,
                               size_t norm_ws_bytes, void* stream) {
  if (n < 0) return fail(ZERO_EINVAL, "zero_reduce_chunks: n %lld < 0", (long long)n);
  if (n_chunks < 1) return fail(ZERO_EINVAL, "zero_reduce_chunks: n_chunks %d < 1", (int)n_chunks);
  if (chunk_stride < n)
    return fail(ZERO_EINVAL, "zero_reduce_chunks: chunk_stride %lld < n %lld", (long long)chunk_stride,
                (long long)n);
  if (!zs::valid_dtype(src_dtype)) return fail(ZERO_EINVAL, "zero_reduce_chunks: bad src_dtype %d", (int)src_dtype);
  if (accumulate != 0 && accumulate != 1) return fail(ZERO_EINVAL, "zero_reduce_chunks: accumulate must be 0 or 1");
  if (!std::isfinite(scale)) return fail(ZERO_EINVAL, "zero_reduce_chunks: non-finite scale");
  if (n > 0 && (d_acc == nullptr || d_chunks == nullptr)) return fail(ZERO_EINVAL, "zero_reduce_chunks: NULL buffer");
  const int64_t es = (src_dtype == ZERO_F32) ? 4 : 2;
  if (chunk_stride > (int64_t(1) << 62) / es / n_chunks)
    return fail(ZERO_EINVAL, "zero_reduce_chunks: %d chunks of %lld elements exceed 2^62 bytes", (int)n_chunks,
                (long long)chunk_stride);
  const zero_status w = check_norm_ws("zero_reduce_chunks", d_norm_ws, norm_ws_bytes, n);
  if (w != ZERO_OK) return w;
  if (n == 0) return ZERO_OK;
  return zs::launch_reduce_chunks(d_acc, d_chunks, src_dtype, n_chunks, chunk_stride, n, scale, d_scale,
                                  accumulate, d_found_nonfinite, static_cast<double*>(d_norm_ws),
                                  zs::as_stream(stream));
}

size_t zero_grad_sqnorm_workspace_bytes(int64_t n) {
  if (n <= 0) return 0;
  return static_cast<size_t>((n + zs::kSqTile - 1) / zs::kSqTile) * sizeof(double);
}

zero_status zero_grad_sqnorm(const float* d_grad, int64_t n, double extra_sqnorm, double max_norm, void* d_ws,
                             size_t ws_bytes, zero_norm_result* d_out, void* stream) {
  if (n < 0) return fail(ZERO_EINVAL, "zero_grad_sqnorm: n %lld < 0", (long long)n);
  if (n > 0 && d_grad == nullptr) return fail(ZERO_EINVAL, "zero_grad_sqnorm: NULL d_grad");
  if (d_out == nullptr) return fail(ZERO_EINVAL, "zero_grad_sqnorm: NULL d_out");
  if (std::isnan(max_norm) || max_norm < 0.0) return fail(ZERO_EINVAL, "zero_grad_sqnorm: bad max_norm");
  if (!std::isfinite(extra_sqnorm) || extra_sqnorm < 0.0)
    return fail(ZERO_EINVAL, "zero_grad_sqnorm: bad extra_sqnorm");
  const size_t need = zero_grad_sqnorm_workspace_bytes(n);
  if (need > 0 && (d_ws == nullptr || ws_bytes < need))
    return fail(ZERO_EINVAL, "zero_grad_sqnorm: workspace %zu bytes < %zu needed", d_ws ? ws_bytes : 0, need);
  if (need > 0 && !zs::aligned(d_ws, 8)) return fail(ZERO_EINVAL, "zero_grad_sqnorm: workspace not 8-byte aligned");
  return zs::launch_sqnorm(d_grad, n, extra_sqnorm, max_norm, static_cast<double*>(d_ws), d_out,
                           zs::as_stream(stream));
}

zero_status zero_grad_sqnorm_finalize(const void* d_ws, int64_t n, double extra_sqnorm, double max_norm,
                                      zero_norm_result* d_out, void* stream) {
  if (n < 0) return fail(ZERO_EINVAL, "zero_grad_sqnorm_finalize: n %lld < 0", (long long)n);
  if (d_out == nullptr) return fail(ZERO_EINVAL, "zero_grad_sqnorm_finalize: NULL d_out");
  if (n > 0 && d_ws == nullptr) return fail(ZERO_EINVAL, "zero_grad_sqnorm_finalize: NULL d_ws");
  if (n > 0 && !zs::aligned(d_ws, 8)) return fail(ZERO_EINVAL, "zero_grad_sqnorm_finalize: d_ws not 8-byte aligned");
  if (std::isnan(max_norm) || max_norm < 0.0) return fail(ZERO_EINVAL, "zero_grad_sqnorm_finalize: bad max_norm");
  if (!std::isfinite(extra_sqnorm) || extra_sqnorm < 0.0)
    return fail(ZERO_EINVAL, "zero_grad_sqnorm_finalize: bad extra_sqnorm");
  return zs::launch_sqnorm_finalize(static_cast<const double*>(d_ws), n, extra_sqnorm, max_norm, d_out,
                                    zs::as_stream(stream));
}

zero_status zero_grad_sqnorm_combine(const double* d_sqnorms, int32_t n_parts, double max_norm,
                                    zero_norm_result* d_out, void* stream) {
  if (n_parts < 1) return fail(ZERO_EINVAL, "zero_grad_sqnorm_combine: n_parts %d < 1", n_parts);
  if (d_sqnorms == nullptr || d_out == nullptr) return fail(ZERO_EINVAL, "zero_grad_sqnorm_combine: NULL pointer");
  if (!zs::aligned(d_sqnorms, 8)) return fail(ZERO_EINVAL, "zero_grad_sqnorm_combine: d_sqnorms not 8-byte aligned");
  if (std::isnan(max_norm) || max_norm < 0.0) return fail(ZERO_EINVAL, "zero_grad_sqnorm_combine: bad max_norm");
  return zs::launch_sqnorm_combine(d_sqnorms, n_parts, max_norm, d_out, zs::as_stream(stream));
}

static zero_status check_loss_scale_policy(const char* who, double growth_factor, double backoff_factor,
                                           int32_t growth_interval) {
  if (!(growth_factor > 1.0) || !std::isfinite(growth_factor))
    return fail(ZERO_EINVAL, "%s: growth_factor must be > 1 and finite", who);
  if (!(backoff_factor > 0.0 && backoff_factor < 1.0))
    return fail(ZERO_EINVAL, "%s: backoff_factor must be in (0, 1)", who);
  if (growth_interval < 1) return fail(ZERO_EINVAL, "%s: growth_interval < 1", who);
  return ZERO_OK;
}

zero_status zero_loss_scale_update(float* scale, int32_t* growth_tracker, int32_t found_inf, double growth_factor,
                                   double backoff_factor, int32_t growth_interval) {
  if (scale == nullptr || growth_tracker == nullptr)
    return fail(ZERO_EINVAL, "zero_loss_scale_update: NULL scale or growth_tracker");
  const zero_status c = check_loss_scale_policy("zero_loss_scale_update", growth_factor, backoff_factor,
                                                growth_interval);
  if (c != ZERO_OK) return c;
  if (found_inf) {
    *scale = static_cast<float>(static_cast<double>(*scale) * backoff_factor);
    *growth_tracker = 0;
    return ZERO_OK;
  }
  const int32_t good = *growth_tracker + 1;
  if (good >= growth_interval) {
    const float grown = static_cast<float>(static_cast<double>(*scale) * growth_factor);
    if (std::isfinite(grown)) *scale = grown;
    *growth_tracker = 0;
  } else {
    *growth_tracker = good;
  }
  return ZERO_OK;
}

zero_status zero_loss_scale_update_device(zero_loss_scale_state* d_state, int32_t accum_steps, double growth_factor,
                                          double backoff_factor, int32_t growth_interval,
                                          const zero_norm_result* d_norm, void* stream) {
  if (d_state == nullptr) return fail(ZERO_EINVAL, "zero_loss_scale_update_device: NULL d_state");
  if (accum_steps < 1) return fail(ZERO_EINVAL, "zero_loss_scale_update_device: accum_steps < 1");
  const zero_status c = check_loss_scale_policy("zero_loss_scale_update_device", growth_factor, backoff_factor,
                                                growth_interval);
  if (c != ZERO_OK) return c;
  return zs::launch_loss_scale_update(d_state, accum_steps, growth_factor, backoff_factor, growth_interval, d_norm,
                                      zs::as_stream(stream));
}

static zero_status adamw_scalars(const char* who, const zero_adamw_hparams* hp, int64_t step, zs::AdamScalars* s) {
  if (hp == nullptr) return fail(ZERO_EINVAL, "%s: NULL hparams", who);
  if (step < 1) return fail(ZERO_EINVAL, "%s: step %lld < 1", who, (long long)step);
  const double lr = hp->lr, b1 = hp->beta1, b2 = hp->beta2, eps = hp->eps, wd = hp->weight_decay;
  if (!(std::isfinite(lr) && lr >= 0.0)) return fail(ZERO_EINVAL, "%s: bad lr", who);
  if (!(b1 >= 0.0 && b1 < 1.0 && b2 >= 0.0 && b2 < 1.0)) return fail(ZERO_EINVAL, "%s: bad betas", who);
  if (!(std::isfinite(eps) && eps > 0.0)) return fail(ZERO_EINVAL, "%s: bad eps", who);
  if (!(std::isfinite(wd) && wd >= 0.0)) return fail(ZERO_EINVAL, "%s: bad weight_decay", who);
  // per-step scalars in binary64, each rounded to binary32 once (the device
  // step state of graph-captured steps uses the same code)
  *s = zs::adam_scalars(lr, b1, b2, eps, wd, step);
  return ZERO_OK;
}

zero_status zero_adamw_scalars(const zero_adamw_hparams* hp, int64_t step, float* out) {
  if (out == nullptr) return fail(ZERO_EINVAL, "zero_adamw_scalars: NULL out");
  zs::AdamScalars s;
  const zero_status st = adamw_scalars("zero_adamw_scalars", hp, step, &s);
  if (st != ZERO_OK) return st;
  const float v[8] = {s.step_size, s.bc2_sqrt, s.decay, s.b1, s.omb1, s.b2, s.omb2, s.eps};
  for (int i = 0; i < 8; ++i) out[i] = v[i];
  return ZERO_OK;
}

zero_status zero_adamw_step(float* d_master, float* d_exp_avg, float* d_exp_avg_sq, const float* d_grad,
                            void* d_param_lowp, zero_dtype lowp_dtype, int64_t n, const zero_adamw_hparams* hp,
                            int64_t step, const zero_norm_result* d_clip, void* stream) {
  if (n < 0) return fail(ZERO_EINVAL, "zero_adamw_step: n %lld < 0", (long long)n);
  zs::AdamScalars s;
  const zero_status hs = adamw_scalars("zero_adamw_step", hp, step, &s);
  if (hs != ZERO_OK) return hs;
  if (n > 0 && (d_master == nullptr || d_exp_avg == nullptr || d_exp_avg_sq == nullptr || d_grad == nullptr))
    return fail(ZERO_EINVAL, "zero_adamw_step: NULL state or grad buffer");
  if (d_param_lowp != nullptr && lowp_dtype != ZERO_BF16 && lowp_dtype != ZERO_F16)
    return fail(ZERO_EINVAL, "zero_adamw_step: lowp_dtype must be BF16 or F16");
  if (n == 0) return ZERO_OK;
  return zs::launch_adamw(d_master, d_exp_avg, d_exp_avg_sq, d_grad, d_param_lowp, lowp_dtype, n, s, nullptr,
                          d_clip, zs::as_stream(stream));
}

zero_status zero_adamw_step_tensors(float* d_master, float* d_exp_avg, float* d_exp_avg_sq,
                                    const zero_tensor* d_table, int32_t n_tensors, int64_t total,
                                    zero_dtype grad_dtype, int64_t shard_start, float grad_scale,
                                    const float* d_grad_scale, const float* d_acc, void* d_param_lowp,
                                    zero_dtype lowp_dtype, int64_t n, const zero_adamw_hparams* hp, int64_t step,
                                    const zero_norm_result* d_clip, void* stream) {
  const char* who = "zero_adamw_step_tensors";
  if (n < 0) return fail(ZERO_EINVAL, "%s: n %lld < 0", who, (long long)n);
  zs::AdamScalars s;
  const zero_status hs = adamw_scalars(who, hp, step, &s);
  if (hs != ZERO_OK) return hs;
  if (n_tensors < 0 || (n_tensors > 0 && d_table == nullptr)) return fail(ZERO_EINVAL, "%s: bad table", who);
  if (total < 0 || (n_tensors == 0 && total != 0)) return fail(ZERO_EINVAL, "%s: total does not fit the table", who);
  if (shard_start < 0 || n > total - shard_start)
    return fail(ZERO_EINVAL, "%s: [%lld, %lld) outside [0, %lld]", who, (long long)shard_start,
                (long long)(shard_start + n), (long long)total);
  if (!zs::valid_dtype(grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", who, (int)grad_dtype);
  if (!std::isfinite(grad_scale)) return fail(ZERO_EINVAL, "%s: non-finite grad_scale", who);
  if (n > 0 && (d_master == nullptr || d_exp_avg == nullptr || d_exp_avg_sq == nullptr))
    return fail(ZERO_EINVAL, "%s: NULL state buffer", who);
  if (d_param_lowp != nullptr && lowp_dtype != ZERO_BF16 && lowp_dtype != ZERO_F16)
    return fail(ZERO_EINVAL, "%s: lowp_dtype must be BF16 or F16", who);
  if (n == 0) return ZERO_OK;
  return zs::launch_adamw_table(d_master, d_exp_avg, d_exp_avg_sq, d_acc, d_table, n_tensors, grad_dtype,
                                shard_start, grad_scale, d_grad_scale, d_param_lowp, lowp_dtype, n, s, nullptr,
                                d_clip, zs::as_stream(stream));
}

// ------------------------------------------------------------- debug builds
zero_status zero_debug_errors(uint64_t* out, int32_t reset) {
  if (out == nullptr) return fail(ZERO_EINVAL, "zero_debug_errors: NULL out");
#ifdef ZERO_DEBUG
  zero_status (*const readers[])(unsigned long long*, bool) = {
      zs::debug_read_adamw,          zs::debug_read_adamw_table,        zs::debug_read_adamw_table_acc,
      zs::debug_read_adamw_table_p4, zs::debug_read_adamw_table_p4_acc, zs::debug_read_adamw_device,
      zs::debug_read_adamw_list,     zs::debug_read_adamw_list8,       zs::debug_read_adamw_table8,
      zs::debug_read_state8,
      zs::debug_read_flatten,        zs::debug_read_sqnorm};
  uint64_t total = 0, first[3] = {0, 0, 0};
  for (auto rd : readers) {
    unsigned long long r[4];
    const zero_status st = rd(r, reset != 0);
    if (st != ZERO_OK) return st;
    if (r[0] != 0 && total == 0) {
      first[0] = r[1];
      first[1] = r[2];
      first[2] = r[3];
    }
    total += r[0];
  }
  out[0] = total;
  out[1] = first[0];
  out[2] = first[1];
  out[3] = first[2];
  return ZERO_OK;
#else
  (void)reset;
  return fail(ZERO_EINVAL, "zero_debug_errors: this library was built without ZERO_DEBUG");
#endif
}

zero_status zero_debug_selftest(int64_t index, void* stream) {
#ifdef ZERO_DEBUG
  return zs::launch_debug_selftest(index, zs::as_stream(stream));
#else
  (void)index;
  (void)stream;
  return fail(ZERO_EINVAL, "zero_debug_selftest: this library was built without ZERO_DEBUG");
#endif
}

// ------------------------------------------------------------- graph-capturable steps
static zero_status check_state(const char* who, const void* d_state) {
  if (d_state == nullptr) return fail(ZERO_EINVAL, "%s: NULL d_state", who);
  if (!zs::aligned(d_state, 8)) return fail(ZERO_EINVAL, "%s: d_state not 8-byte aligned", who);
  return ZERO_OK;
}

zero_status zero_adamw_prepare_device(const zero_adamw_hparams* d_hp, const zero_norm_result* d_clip,
                                      zero_adamw_device_state* d_state, void* stream) {
  const char* who = "zero_adamw_prepare_device";
  if (d_hp == nullptr) return fail(ZERO_EINVAL, "%s: NULL d_hp", who);
  if (!zs::aligned(d_hp, 8)) return fail(ZERO_EINVAL, "%s: d_hp not 8-byte aligned", who);
  const zero_status c = check_state(who, d_state);
  if (c != ZERO_OK) return c;
  return zs::launch_adamw_prepare(d_hp, d_clip, d_state, zs::as_stream(stream));
}

zero_status zero_adamw_step_device(float* d_master, float* d_exp_avg, float* d_exp_avg_sq, const float* d_grad,
                                   void* d_param_lowp, zero_dtype lowp_dtype, int64_t n,
                                   const zero_adamw_device_state* d_state, const zero_norm_result* d_clip,
                                   void* stream) {
  const char* who = "zero_adamw_step_device";
  if (n < 0) return fail(ZERO_EINVAL, "%s: n %lld < 0", who, (long long)n);
  const zero_status c = check_state(who, d_state);
  if (c != ZERO_OK) return c;
  if (n > 0 && (d_master == nullptr || d_exp_avg == nullptr || d_exp_avg_sq == nullptr || d_grad == nullptr))
    return fail(ZERO_EINVAL, "%s: NULL state or grad buffer", who);
  if (d_param_lowp != nullptr && lowp_dtype != ZERO_BF16 && lowp_dtype != ZERO_F16)
    return fail(ZERO_EINVAL, "%s: lowp_dtype must be BF16 or F16", who);
  if (n == 0) return ZERO_OK;
  return zs::launch_adamw(d_master, d_exp_avg, d_exp_avg_sq, d_grad, d_param_lowp, lowp_dtype, n, zs::AdamScalars{},
                          d_state, d_clip, zs::as_stream(stream));
}

zero_status zero_adamw_step_tensors_device(float* d_master, float* d_exp_avg, float* d_exp_avg_sq,
                                           const zero_tensor* d_table, int32_t n_tensors, int64_t total,
                                           zero_dtype grad_dtype, int64_t shard_start, float grad_scale,
                                           const float* d_grad_scale, const float* d_acc, void* d_param_lowp,
                                           zero_dtype lowp_dtype, int64_t n, const zero_adamw_device_state* d_state,
                                           const zero_norm_result* d_clip, void* stream) {
  const char* who = "zero_adamw_step_tensors_device";
  if (n < 0) return fail(ZERO_EINVAL, "%s: n %lld < 0", who, (long long)n);
  const zero_status c = check_state(who, d_state);
  if (c != ZERO_OK) return c;
  if (n_tensors < 0 || (n_tensors > 0 && d_table == nullptr)) return fail(ZERO_EINVAL, "%s: bad table", who);
  if (total < 0 || (n_tensors == 0 && total != 0)) return fail(ZERO_EINVAL, "%s: total does not fit the table", who);
  if (shard_start < 0 || n > total - shard_start)
    return fail(ZERO_EINVAL, "%s: [%lld, %lld) outside [0, %lld]", who, (long long)shard_start,
                (long long)(shard_start + n), (long long)total);
  if (!zs::valid_dtype(grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", who, (int)grad_dtype);
  if (!std::isfinite(grad_scale)) return fail(ZERO_EINVAL, "%s: non-finite grad_scale", who);
  if (n > 0 && (d_master == nullptr || d_exp_avg == nullptr || d_exp_avg_sq == nullptr))
    return fail(ZERO_EINVAL, "%s: NULL state buffer", who);
  if (d_param_lowp != nullptr && lowp_dtype != ZERO_BF16 && lowp_dtype != ZERO_F16)
    return fail(ZERO_EINVAL, "%s: lowp_dtype must be BF16 or F16", who);
  if (n == 0) return ZERO_OK;
  return zs::launch_adamw_table(d_master, d_exp_avg, d_exp_avg_sq, d_acc, d_table, n_tensors, grad_dtype,
                                shard_start, grad_scale, d_grad_scale, d_param_lowp, lowp_dtype, n,
                                zs::AdamScalars{}, d_state, d_clip, zs::as_stream(stream));
}

// ------------------------------------------------- 8-bit moments, tensor lists
static zero_status check_state8(const char* who, const zero_state8* q, int64_t n) {
  if (n < 0) return fail(ZERO_EINVAL, "%s: n %lld < 0", who, (long long)n);
  if (q == nullptr) return fail(ZERO_EINVAL, "%s: NULL 8-bit state", who);
  if (n > 0 && (q->exp_avg == nullptr || q->exp_avg_scale == nullptr || q->root == nullptr || q->root_scale == nullptr))
    return fail(ZERO_EINVAL, "%s: NULL 8-bit state buffer", who);
  if (!zs::aligned(q->exp_avg_scale, 4) || !zs::aligned(q->root_scale, 4))
    return fail(ZERO_EINVAL, "%s: scales not 4-byte aligned", who);
  return ZERO_OK;
}

zero_status zero_state8_pack(const float* d_exp_avg, const float* d_exp_avg_sq, int64_t n, const zero_state8* q,
                             void* stream) {
  const zero_status c = check_state8("zero_state8_pack", q, n);
  if (c != ZERO_OK) return c;
  if (n == 0) return ZERO_OK;
  if (d_exp_avg == nullptr || d_exp_avg_sq == nullptr) return fail(ZERO_EINVAL, "zero_state8_pack: NULL buffer");
  return zs::launch_state8_pack(d_exp_avg, d_exp_avg_sq, n, *q, zs::as_stream(stream));
}

zero_status zero_state8_unpack(const zero_state8* q, int64_t n, float* d_exp_avg, float* d_exp_avg_sq, void* stream) {
  const zero_status c = check_state8("zero_state8_unpack", q, n);
  if (c != ZERO_OK) return c;
  if (n == 0) return ZERO_OK;
  if (d_exp_avg == nullptr || d_exp_avg_sq == nullptr) return fail(ZERO_EINVAL, "zero_state8_unpack: NULL buffer");
  return zs::launch_state8_unpack(*q, n, d_exp_avg, d_exp_avg_sq, zs::as_stream(stream));
}

static zero_status check_rounding(const char* who, const zero_rounding* r) {
  if (r == nullptr) return ZERO_OK;
  if (r->root_bits != 0 && r->root_bits != 7 && r->root_bits != 16)
    return fail(ZERO_EINVAL, "%s: root_bits %d, not 0, 7 or 16", who, (int)r->root_bits);
  if (r->reserved != 0) return fail(ZERO_EINVAL, "%s: rounding's reserved != 0", who);
  return ZERO_OK;
}

static zero_status step8_tensors(const char* who, float* d_master, const zero_state8* q, const zero_tensor* d_table,
                                 int32_t n_tensors, int64_t total, zero_dtype grad_dtype, int64_t shard_start,
                                 float grad_scale, const float* d_grad_scale, const float* d_acc, void* d_param_lowp,
                                 zero_dtype lowp_dtype, int64_t n, const zs::AdamScalars& s, int64_t step,
                                 const zero_adamw_device_state* d_state, const zero_rounding* rounding,
                                 const zero_norm_result* d_clip, void* stream) {
  const zero_status c = check_state8(who, q, n);
  if (c != ZERO_OK) return c;
  if (n_tensors < 0 || (n_tensors > 0 && d_table == nullptr)) return fail(ZERO_EINVAL, "%s: bad table", who);
  if (total < 0 || (n_tensors == 0 && total != 0)) return fail(ZERO_EINVAL, "%s: total does not fit the table", who);
  if (shard_start < 0 || n > total - shard_start)
    return fail(ZERO_EINVAL, "%s: [%lld, %lld) outside [0, %lld]", who, (long long)shard_start,
                (long long)(shard_start + n), (long long)total);
  if (!zs::valid_dtype(grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", who, (int)grad_dtype);
  if (!std::isfinite(grad_scale)) return fail(ZERO_EINVAL, "%s: non-finite grad_scale", who);
  if (n > 0 && d_master == nullptr) return fail(ZERO_EINVAL, "%s: NULL master", who);
  if (n / 2048 >= INT32_MAX) return fail(ZERO_EINVAL, "%s: n %lld exceeds 2^42", who, (long long)n);
  if (d_param_lowp != nullptr && lowp_dtype != ZERO_BF16 && lowp_dtype != ZERO_F16)
    return fail(ZERO_EINVAL, "%s: lowp_dtype must be BF16 or F16", who);
  const zero_status r = check_rounding(who, rounding);
  if (r != ZERO_OK) return r;
  if (n == 0) return ZERO_OK;
  const zs::Table8Args a{d_master, *q, d_acc, d_table, n_tensors, grad_dtype, shard_start, n, grad_scale, d_grad_scale,
                         d_param_lowp, lowp_dtype, d_state,
                         d_state == nullptr ? zs::rounding_base(rounding, &step, zs::Betas{s.b1, s.b2, s.b2})
                                            : zs::rounding_base(rounding, nullptr, zs::Betas{}),
                         d_clip};
  return zs::launch_adamw_table8(a, s, zs::as_stream(stream));
}

zero_status zero_adamw_step8_tensors(float* d_master, const zero_state8* q, const zero_tensor* d_table,
                                     int32_t n_tensors, int64_t total, zero_dtype grad_dtype, int64_t shard_start,
                                     float grad_scale, const float* d_grad_scale, const float* d_acc,
                                     void* d_param_lowp, zero_dtype lowp_dtype, int64_t n,
                                     const zero_adamw_hparams* hp, int64_t step, const zero_rounding* rounding,
                                     const zero_norm_result* d_clip, void* stream) {
  const char* who = "zero_adamw_step8_tensors";
  zs::AdamScalars s;
  const zero_status hs = adamw_scalars(who, hp, step, &s);
  if (hs != ZERO_OK) return hs;
  return step8_tensors(who, d_master, q, d_table, n_tensors, total, grad_dtype, shard_start, grad_scale, d_grad_scale,
                       d_acc, d_param_lowp, lowp_dtype, n, s, step, nullptr, rounding, d_clip, stream);
}

zero_status zero_adamw_step8_tensors_device(float* d_master, const zero_state8* q, const zero_tensor* d_table,
                                            int32_t n_tensors, int64_t total, zero_dtype grad_dtype,
                                            int64_t shard_start, float grad_scale, const float* d_grad_scale,
                                            const float* d_acc, void* d_param_lowp, zero_dtype lowp_dtype, int64_t n,
                                            const zero_adamw_device_state* d_state, const zero_rounding* rounding,
                                            const zero_norm_result* d_clip, void* stream) {
  const char* who = "zero_adamw_step8_tensors_device";
  const zero_status c = check_state(who, d_state);
  if (c != ZERO_OK) return c;
  return step8_tensors(who, d_master, q, d_table, n_tensors, total, grad_dtype, shard_start, grad_scale, d_grad_scale,
                       d_acc, d_param_lowp, lowp_dtype, n, zs::AdamScalars{}, 0, d_state, rounding, d_clip,
                       stream);
}

static zero_status check_groups(const char* who, int32_t n_groups) {
  if (n_groups < 1 || n_groups > ZERO_LIST_MAX_GROUPS)
    return fail(ZERO_EINVAL, "%s: %d groups, not 1 to %d", who, (int)n_groups, ZERO_LIST_MAX_GROUPS);
  return ZERO_OK;
}

zero_status zero_list_chunks(const zero_list_tensor* list, int32_t n_tensors, int32_t n_groups, int32_t state_bits,
                             int32_t* first_chunk, int32_t* n_chunks) {
  const char* who = "zero_list_chunks";
  if (n_tensors < 0 || (n_tensors > 0 && list == nullptr)) return fail(ZERO_EINVAL, "%s: bad list", who);
  const zero_status g = check_groups(who, n_groups);
  if (g != ZERO_OK) return g;
  if (state_bits != 32 && state_bits != 8) return fail(ZERO_EINVAL, "%s: state_bits must be 32 or 8", who);
  int64_t count = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const zero_list_tensor& t = list[i];
    if (t.numel < 0) return fail(ZERO_EINVAL, "%s: numel[%d] = %lld < 0", who, (int)i, (long long)t.numel);
    if (t.group < 0 || t.group >= n_groups)
      return fail(ZERO_EINVAL, "%s: group[%d] = %d of %d", who, (int)i, (int)t.group, (int)n_groups);
    if (t.reserved != 0) return fail(ZERO_EINVAL, "%s: reserved[%d] != 0", who, (int)i);
    if (t.numel > 0 && (t.master == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr))
      return fail(ZERO_EINVAL, "%s: NULL buffer of tensor %d", who, (int)i);
    const bool fits = state_bits == 32 ? t.exp_avg_scale == nullptr && t.root_scale == nullptr
                                       : t.exp_avg_scale != nullptr && t.root_scale != nullptr;
    if (t.numel > 0 && !fits)
      return fail(ZERO_EINVAL, "%s: the scales of tensor %d do not fit %d-bit states", who, (int)i, (int)state_bits);
    const uintptr_t sa = state_bits == 32 ? 4 : 1;
    if (!zs::aligned(t.master, 4) || !zs::aligned(t.exp_avg, sa) || !zs::aligned(t.exp_avg_sq, sa) ||
        !zs::aligned(t.exp_avg_scale, 4) || !zs::aligned(t.root_scale, 4) || !zs::aligned(t.lowp, 2))
      return fail(ZERO_EINVAL, "%s: a buffer of tensor %d is not aligned to its elements", who, (int)i);
    if (first_chunk != nullptr) first_chunk[i] = static_cast<int32_t>(count);
    count += t.numel / zs::kListChunk + (t.numel % zs::kListChunk != 0 ? 1 : 0);
    if (count > INT32_MAX) return fail(ZERO_EINVAL, "%s: 2^31 chunks or more up to tensor %d", who, (int)i);
  }
  if (first_chunk != nullptr) first_chunk[n_tensors] = static_cast<int32_t>(count);
  if (n_chunks != nullptr) *n_chunks = static_cast<int32_t>(count);
  return ZERO_OK;
}

// The checks and the launch that both forms of the list step share.
static zero_status adamw_list(const char* who, const zs::ListArgs& a, const zs::ListScalars& s, int32_t n_groups,
                              void* stream) {
  if (a.n_tensors < 0 || a.n_chunks < 0) return fail(ZERO_EINVAL, "%s: n_tensors or n_chunks < 0", who);
  if (a.n_chunks > 0 && (a.list == nullptr || a.first_chunk == nullptr || a.grads == nullptr || a.n_tensors == 0))
    return fail(ZERO_EINVAL, "%s: NULL list, first_chunk or grads", who);
  if (!zs::aligned(a.list, 8) || !zs::aligned(a.first_chunk, 4) || !zs::aligned(a.grads, 8))
    return fail(ZERO_EINVAL, "%s: list, first_chunk or grads not aligned", who);
  const zero_status g = check_groups(who, n_groups);
  if (g != ZERO_OK) return g;
  if (a.state_bits != 32 && a.state_bits != 8) return fail(ZERO_EINVAL, "%s: state_bits must be 32 or 8", who);
  if (a.rounding.how != zs::kNearest && a.state_bits == 32)
    return fail(ZERO_EINVAL, "%s: a rounding seed needs 8-bit states", who);
  if (!zs::valid_dtype(a.grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", who, a.grad_dtype);
  if (a.lowp_dtype != ZERO_BF16 && a.lowp_dtype != ZERO_F16)
    return fail(ZERO_EINVAL, "%s: lowp_dtype must be BF16 or F16", who);
  if (!std::isfinite(a.gscale)) return fail(ZERO_EINVAL, "%s: non-finite grad_scale", who);
  if (a.n_chunks == 0) return ZERO_OK;
  return zs::launch_adamw_list(a, s, zs::as_stream(stream));
}

zero_status zero_adamw_list(const zero_list_tensor* d_list, int32_t n_tensors, const int32_t* d_first_chunk,
                            int32_t n_chunks, int32_t state_bits, const zero_tensor* d_grads, zero_dtype grad_dtype,
                            float grad_scale, const float* d_grad_scale, zero_dtype lowp_dtype,
                            const zero_adamw_hparams* groups, int32_t n_groups, int64_t step,
                            const zero_rounding* rounding, const zero_norm_result* d_clip, void* stream) {
  const char* who = "zero_adamw_list";
  const zero_status g = check_groups(who, n_groups);
  if (g != ZERO_OK) return g;
  if (groups == nullptr) return fail(ZERO_EINVAL, "%s: NULL groups", who);
  const zero_status r = check_rounding(who, rounding);
  if (r != ZERO_OK) return r;
  zs::ListScalars s{};
  zs::Betas b{0.0f, 1.0f, 0.0f};
  for (int32_t i = 0; i < n_groups; ++i) {
    const zero_status hs = adamw_scalars(who, &groups[i], step, &s.s[i]);
    if (hs != ZERO_OK) return hs;
    b.beta1 = std::max(b.beta1, s.s[i].b1);
    b.least2 = std::min(b.least2, s.s[i].b2);
    b.most2 = std::max(b.most2, s.s[i].b2);
  }
  const zs::ListArgs a{d_list, n_tensors, d_first_chunk, n_chunks, state_bits, d_grads, grad_dtype, grad_scale, d_grad_scale,
                       lowp_dtype, nullptr, zs::rounding_base(rounding, &step, b), d_clip};
  return adamw_list(who, a, s, n_groups, stream);
}

zero_status zero_adamw_list_device(const zero_list_tensor* d_list, int32_t n_tensors, const int32_t* d_first_chunk,
                                   int32_t n_chunks, int32_t state_bits, const zero_tensor* d_grads,
                                   zero_dtype grad_dtype, float grad_scale, const float* d_grad_scale,
                                   zero_dtype lowp_dtype, const zero_adamw_device_state* d_states, int32_t n_groups,
                                   const zero_rounding* rounding, const zero_norm_result* d_clip, void* stream) {
  const char* who = "zero_adamw_list_device";
  const zero_status c = check_state(who, d_states);
  if (c != ZERO_OK) return c;
  const zero_status r = check_rounding(who, rounding);
  if (r != ZERO_OK) return r;
  const zs::ListArgs a{d_list, n_tensors, d_first_chunk, n_chunks, state_bits, d_grads, grad_dtype, grad_scale, d_grad_scale,
                       lowp_dtype, d_states, zs::rounding_base(rounding, nullptr, zs::Betas{}), d_clip};
  return adamw_list(who, a, zs::ListScalars{}, n_groups, stream);
}

zero_status zero_adamw_prepare_list_device(const zero_adamw_hparams* d_hp, int32_t n_groups,
                                           const zero_norm_result* d_clip, zero_adamw_device_state* d_states,
                                           void* stream) {
  const char* who = "zero_adamw_prepare_list_device";
  const zero_status g = check_groups(who, n_groups);
  if (g != ZERO_OK) return g;
  if (d_hp == nullptr) return fail(ZERO_EINVAL, "%s: NULL d_hp", who);
  if (!zs::aligned(d_hp, 8)) return fail(ZERO_EINVAL, "%s: d_hp not 8-byte aligned", who);
  const zero_status c = check_state(who, d_states);
  if (c != ZERO_OK) return c;
  return zs::launch_adamw_prepare_list(d_hp, n_groups, d_clip, d_states, zs::as_stream(stream));
}

}  // extern "C"
