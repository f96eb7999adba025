// extern "C" entry points: argument validation, then the launchers.
// Validation never touches the device, so every error path here can be
// exercised without a GPU.
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/ssmq.h"
#include "internal.h"

namespace {

thread_local char g_err[512] = "";

ssmq_status fail(ssmq_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

// One NVTX range per entry-point call (named after the entry point), seen by
// profilers as the host-side span of the call; a no-op without a tool.
struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

bool aligned16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Host-side fault injection for tests of the error path: when the
// environment variable SSMQ_FAULT_INJECT names an entry point (or "all"),
// that entry point reports a launch failure instead of launching.
bool injected(const char* name) {
  const char* v = getenv("SSMQ_FAULT_INJECT");
  if (!v || !*v) return false;
  return strcmp(v, "all") == 0 || strcmp(v, name) == 0;
}

ssmq_status finish(cudaError_t e, const char* name) {
  if (e != cudaSuccess) return fail(SSMQ_ERR_CUDA, "%s: CUDA error %d (%s)", name, (int)e,
                                    cudaGetErrorString(e));
  return SSMQ_OK;
}

#define REQUIRE(cond, code, ...)        \
  do {                                  \
    if (!(cond)) return fail(code, __VA_ARGS__); \
  } while (0)

ssmq_status check_x(int32_t fmt, const void* x, const int32_t* x_group, const float* x_scale,
                    int32_t n_x_groups, int32_t log2_ratio, const char* fn,
                    bool allow_f16 = false) {
  REQUIRE(fmt >= SSMQ_X_INT8_GROUP && fmt <= SSMQ_X_F16_SOFTEDGE, SSMQ_ERR_INVALID_ARG,
          "%s: x_format %d is not an ssmq_x_format", fn, fmt);
  REQUIRE(allow_f16 || fmt == SSMQ_X_INT8_GROUP || fmt == SSMQ_X_SOFTEDGE, SSMQ_ERR_UNSUPPORTED,
          "%s: binary16 x (x_format %d) is accepted by the Mamba-1 scan only", fn, fmt);
  REQUIRE(x != nullptr, SSMQ_ERR_INVALID_ARG, "%s: x is NULL", fn);
  if (fmt == SSMQ_X_INT8_GROUP || fmt == SSMQ_X_F16_GROUP) {
    REQUIRE(x_group && x_scale, SSMQ_ERR_INVALID_ARG, "%s: x_group / x_scale is NULL", fn);
    REQUIRE(n_x_groups >= 1, SSMQ_ERR_INVALID_ARG, "%s: n_x_groups must be >= 1", fn);
  } else {
    REQUIRE(log2_ratio >= 0 && log2_ratio <= 8, SSMQ_ERR_INVALID_ARG,
            "%s: se_log2_ratio must be in [0, 8]", fn);
  }
  return SSMQ_OK;
}

// optional int8 output: the cluster map and scales come with it
ssmq_status check_yq(const int8_t* y_q, const int32_t* y_group, const float* y_scale,
                     int32_t n_y_groups, const char* fn) {
  if (!y_q) return SSMQ_OK;
  REQUIRE(aligned16(y_q), SSMQ_ERR_ALIGNMENT, "%s: y_q must be 16-byte aligned", fn);
  REQUIRE(y_group && y_scale && n_y_groups >= 1, SSMQ_ERR_INVALID_ARG,
          "%s: y_q needs y_group, y_scale and n_y_groups >= 1", fn);
  return SSMQ_OK;
}

ssmq_status check_src(const void* src, ssmq_dtype dtype, int64_t n, const char* fn) {
  REQUIRE(dtype == SSMQ_F32 || dtype == SSMQ_F16, SSMQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
  REQUIRE(n >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  if (n > 0) REQUIRE(src != nullptr, SSMQ_ERR_INVALID_ARG, "%s: src is NULL", fn);
  return SSMQ_OK;
}

ssmq_status check_ws(void* workspace, size_t ws_bytes, const char* fn) {
  REQUIRE(workspace && ws_bytes >= ssmq::percentile_workspace_bytes(), SSMQ_ERR_INVALID_ARG,
          "%s: workspace of %zu bytes required (got %zu)", fn,
          ssmq::percentile_workspace_bytes(), ws_bytes);
  REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, SSMQ_ERR_ALIGNMENT,
          "%s: workspace must be 256-byte aligned", fn);
  return SSMQ_OK;
}

ssmq_status check_pct_q(const double* q, int32_t nq, const float* out, const char* fn) {
  REQUIRE(q && out && nq >= 1 && nq <= ssmq::percentile_max_q(), SSMQ_ERR_INVALID_ARG,
          "%s: need 1 <= nq <= %d percentiles and out", fn, ssmq::percentile_max_q());
  for (int i = 0; i < nq; ++i)
    REQUIRE(q[i] >= 0.0 && q[i] <= 100.0, SSMQ_ERR_INVALID_ARG,
            "%s: percentile %d outside [0, 100]", fn, i);
  return SSMQ_OK;
}

ssmq_status check_se_cal(double q_lo, double q_hi, float alpha, const float* thresholds,
                         const char* fn) {
  REQUIRE(thresholds != nullptr, SSMQ_ERR_INVALID_ARG, "%s: thresholds is NULL", fn);
  REQUIRE(q_lo >= 0.0 && q_lo <= q_hi && q_hi <= 100.0, SSMQ_ERR_INVALID_ARG,
          "%s: need 0 <= q_lo <= q_hi <= 100", fn);
  REQUIRE(alpha > 0.0f && alpha <= 1.0f, SSMQ_ERR_INVALID_ARG, "%s: alpha must be in (0, 1]", fn);
  return SSMQ_OK;
}

#define CHECK(call)                     \
  do {                                  \
    const ssmq_status s_ = (call);      \
    if (s_ != SSMQ_OK) return s_;       \
  } while (0)

}  // namespace

extern "C" {

const char* ssmq_last_error(void) { return g_err; }

int32_t ssmq_version(void) { return 100; }

ssmq_status ssmq_quantize_groups(const void* src, ssmq_dtype dtype, int64_t outer, int64_t mid,
                                 int64_t inner, const int32_t* group_of_mid, int32_t n_groups,
                                 ssmq_scale_mode mode, float* scales, int8_t* q_out,
                                 uint32_t* status, void* stream) {
  const char* fn = "ssmq_quantize_groups";
  Range nvtx_range(fn);
  REQUIRE(dtype == SSMQ_F32 || dtype == SSMQ_F16, SSMQ_ERR_INVALID_ARG, "%s: bad dtype %d", fn,
          (int)dtype);
  REQUIRE(mode == SSMQ_SCALE_STATIC || mode == SSMQ_SCALE_ABSMAX, SSMQ_ERR_INVALID_ARG,
          "%s: bad scale mode %d", fn, (int)mode);
  REQUIRE(outer >= 0 && mid >= 0 && inner >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  REQUIRE(n_groups >= 1, SSMQ_ERR_INVALID_ARG, "%s: n_groups must be >= 1", fn);
  REQUIRE(scales != nullptr, SSMQ_ERR_INVALID_ARG, "%s: scales is NULL", fn);
  const bool empty = outer == 0 || mid == 0 || inner == 0;
  if (!empty) {
    REQUIRE(src && q_out && group_of_mid, SSMQ_ERR_INVALID_ARG, "%s: NULL tensor", fn);
    REQUIRE(outer <= (INT64_MAX / mid) / inner, SSMQ_ERR_INVALID_ARG, "%s: size overflow", fn);
  }
  REQUIRE(aligned16(src) && aligned16(q_out), SSMQ_ERR_ALIGNMENT,
          "%s: src and q_out must be 16-byte aligned", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  if (empty && mode == SSMQ_SCALE_STATIC) return SSMQ_OK;
  return finish(ssmq::launch_quantize(src, dtype == SSMQ_F16, empty ? 0 : outer, mid, inner,
                                      group_of_mid, n_groups, mode == SSMQ_SCALE_ABSMAX, scales,
                                      q_out, status, (cudaStream_t)stream),
                fn);
}

ssmq_status ssmq_quantize_groups_batch(const ssmq_quant_job* jobs, int32_t n_jobs,
                                       uint32_t* status, void* stream) {
  const char* fn = "ssmq_quantize_groups_batch";
  Range nvtx_range(fn);
  REQUIRE(jobs != nullptr, SSMQ_ERR_INVALID_ARG, "%s: jobs is NULL", fn);
  REQUIRE(n_jobs >= 1 && n_jobs <= ssmq::kMaxQuantJobs, SSMQ_ERR_INVALID_ARG,
          "%s: n_jobs must be in [1, %d] (got %d)", fn, ssmq::kMaxQuantJobs, (int)n_jobs);
  ssmq::QuantJob hj[ssmq::kMaxQuantJobs];
  for (int k = 0; k < n_jobs; ++k) {
    const ssmq_quant_job& j = jobs[k];
    REQUIRE(j.dtype == SSMQ_F32 || j.dtype == SSMQ_F16, SSMQ_ERR_INVALID_ARG,
            "%s: job %d: bad dtype %d", fn, k, (int)j.dtype);
    REQUIRE(j.outer >= 0 && j.mid >= 0 && j.inner >= 0, SSMQ_ERR_INVALID_ARG,
            "%s: job %d: negative size", fn, k);
    REQUIRE(j.n_groups >= 1, SSMQ_ERR_INVALID_ARG, "%s: job %d: n_groups must be >= 1", fn, k);
    REQUIRE(j.scales != nullptr, SSMQ_ERR_INVALID_ARG, "%s: job %d: scales is NULL", fn, k);
    const bool empty = j.outer == 0 || j.mid == 0 || j.inner == 0;
    if (!empty) {
      REQUIRE(j.src && j.q_out && j.group_of_mid, SSMQ_ERR_INVALID_ARG, "%s: job %d: NULL tensor",
              fn, k);
      REQUIRE(j.outer <= (INT64_MAX / j.mid) / j.inner, SSMQ_ERR_INVALID_ARG,
              "%s: job %d: size overflow", fn, k);
    }
    REQUIRE(aligned16(j.src) && aligned16(j.q_out), SSMQ_ERR_ALIGNMENT,
            "%s: job %d: src and q_out must be 16-byte aligned", fn, k);
    hj[k] = ssmq::QuantJob{j.src, j.dtype == SSMQ_F16, empty ? 0 : j.outer, j.mid, j.inner,
                           j.group_of_mid, j.n_groups, j.scales, j.q_out};
  }
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_quantize_batch(hj, n_jobs, status, (cudaStream_t)stream), fn);
}

ssmq_status ssmq_softedge_encode(const void* src, ssmq_dtype dtype, int64_t n, float scale,
                                 float thr_lo, float thr_hi, int32_t log2_ratio, uint8_t* codes,
                                 uint32_t* status, void* stream) {
  const char* fn = "ssmq_softedge_encode";
  Range nvtx_range(fn);
  REQUIRE(dtype == SSMQ_F32 || dtype == SSMQ_F16, SSMQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
  REQUIRE(n >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  REQUIRE(thr_lo <= thr_hi, SSMQ_ERR_INVALID_ARG,
          "%s: thr_lo must not exceed thr_hi (got %g > %g)", fn, (double)thr_lo, (double)thr_hi);
  REQUIRE(log2_ratio >= 0 && log2_ratio <= 8, SSMQ_ERR_INVALID_ARG,
          "%s: log2_ratio must be in [0, 8]", fn);
  if (n > 0) REQUIRE(src && codes, SSMQ_ERR_INVALID_ARG, "%s: NULL tensor", fn);
  REQUIRE(aligned16(src) && aligned16(codes), SSMQ_ERR_ALIGNMENT, "%s: 16-byte alignment", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_softedge_encode(src, dtype == SSMQ_F16, n, scale, thr_lo, thr_hi,
                                             log2_ratio, codes, status, (cudaStream_t)stream),
                fn);
}

ssmq_status ssmq_group_absmax(const void* src, ssmq_dtype dtype, int64_t outer, int64_t mid,
                              int64_t inner, const int32_t* group_of_mid, int32_t n_groups,
                              float* absmax, uint32_t* status, void* stream) {
  const char* fn = "ssmq_group_absmax";
  Range nvtx_range(fn);
  REQUIRE(dtype == SSMQ_F32 || dtype == SSMQ_F16, SSMQ_ERR_INVALID_ARG, "%s: bad dtype %d", fn,
          (int)dtype);
  REQUIRE(outer >= 0 && mid >= 0 && inner >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  REQUIRE(n_groups >= 1 && absmax, SSMQ_ERR_INVALID_ARG, "%s: need n_groups >= 1 and absmax", fn);
  const int64_t n = outer * mid * inner;
  if (n > 0) REQUIRE(src && group_of_mid, SSMQ_ERR_INVALID_ARG, "%s: NULL tensor", fn);
  REQUIRE(aligned16(src), SSMQ_ERR_ALIGNMENT, "%s: src must be 16-byte aligned", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_group_absmax(src, dtype == SSMQ_F16, outer, mid, inner,
                                          group_of_mid, n_groups, absmax, status,
                                          (cudaStream_t)stream),
                fn);
}

ssmq_status ssmq_cluster_by_absmax(const float* absmax, int64_t n, int32_t k, int32_t* cluster_of,
                                   float* scales, uint32_t* status, void* stream) {
  const char* fn = "ssmq_cluster_by_absmax";
  Range nvtx_range(fn);
  REQUIRE(n >= 1 && k >= 1 && k <= n, SSMQ_ERR_INVALID_ARG, "%s: need 1 <= k <= n", fn);
  REQUIRE(n <= 65536, SSMQ_ERR_UNSUPPORTED, "%s: n > 65536 channels", fn);
  REQUIRE(absmax && cluster_of && scales, SSMQ_ERR_INVALID_ARG, "%s: NULL tensor", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_cluster_by_absmax(absmax, (int)n, k, cluster_of, scales, status,
                                               (cudaStream_t)stream),
                fn);
}

ssmq_status ssmq_probe_ex2(int32_t iters, float* sink, int64_t* n_ex2, void* stream) {
  const char* fn = "ssmq_probe_ex2";
  Range nvtx_range(fn);
  REQUIRE(iters >= 1 && sink && n_ex2, SSMQ_ERR_INVALID_ARG,
          "%s: iters >= 1, sink and n_ex2 required", fn);
  REQUIRE(aligned16(sink), SSMQ_ERR_ALIGNMENT, "%s: sink must be 16-byte aligned", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_probe_ex2(iters, sink, n_ex2, (cudaStream_t)stream), fn);
}

size_t ssmq_percentile_workspace_size(void) { return ssmq::percentile_workspace_bytes(); }


ssmq_status ssmq_percentile_abs(const void* src, ssmq_dtype dtype, int64_t n, const double* q,
                                int32_t nq, float* out, void* workspace, size_t ws_bytes,
                                void* stream) {
  const char* fn = "ssmq_percentile_abs";
  Range nvtx_range(fn);
  CHECK(check_src(src, dtype, n, fn));
  CHECK(check_pct_q(q, nq, out, fn));
  CHECK(check_ws(workspace, ws_bytes, fn));
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_percentile_abs(src, dtype == SSMQ_F16, n, q, nq, out, nullptr, 1.0f,
                                            workspace, (cudaStream_t)stream),
                fn);
}

ssmq_status ssmq_softedge_calibrate(const void* src, ssmq_dtype dtype, int64_t n, double q_lo,
                                    double q_hi, float alpha, float* thresholds, void* workspace,
                                    size_t ws_bytes, void* stream) {
  const char* fn = "ssmq_softedge_calibrate";
  Range nvtx_range(fn);
  CHECK(check_src(src, dtype, n, fn));
  CHECK(check_se_cal(q_lo, q_hi, alpha, thresholds, fn));
  CHECK(check_ws(workspace, ws_bytes, fn));
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  const double q[2] = {q_lo, q_hi};
  return finish(ssmq::launch_percentile_abs(src, dtype == SSMQ_F16, n, q, 2,
                                            ssmq::percentile_scratch_out(workspace), thresholds,
                                            alpha, workspace, (cudaStream_t)stream),
                fn);
}

namespace {
// the library's static scratch of the current device, or an error status
ssmq_status static_scratch(void** ws, const char* fn) {
  cudaError_t e;
  const size_t need = ssmq::percentile_workspace_bytes();
  *ws = ssmq::percentile_static_scratch(need, &e);
  REQUIRE(e == cudaSuccess, SSMQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  REQUIRE(*ws != nullptr, SSMQ_ERR_UNSUPPORTED, "%s: %zu bytes of scratch exceed the static array",
          fn, need);
  return SSMQ_OK;
}
}  // namespace

ssmq_status ssmq_percentile_abs_noalloc(const void* src, ssmq_dtype dtype, int64_t n,
                                        const double* q, int32_t nq, float* out, void* stream) {
  const char* fn = "ssmq_percentile_abs_noalloc";
  Range nvtx_range(fn);
  CHECK(check_src(src, dtype, n, fn));  // argument errors before any device call
  CHECK(check_pct_q(q, nq, out, fn));
  void* ws = nullptr;
  CHECK(static_scratch(&ws, fn));
  return ssmq_percentile_abs(src, dtype, n, q, nq, out, ws, ssmq::percentile_workspace_bytes(),
                             stream);
}

ssmq_status ssmq_softedge_calibrate_noalloc(const void* src, ssmq_dtype dtype, int64_t n,
                                            double q_lo, double q_hi, float alpha,
                                            float* thresholds, void* stream) {
  const char* fn = "ssmq_softedge_calibrate_noalloc";
  Range nvtx_range(fn);
  CHECK(check_src(src, dtype, n, fn));
  CHECK(check_se_cal(q_lo, q_hi, alpha, thresholds, fn));
  void* ws = nullptr;
  CHECK(static_scratch(&ws, fn));
  return ssmq_softedge_calibrate(src, dtype, n, q_lo, q_hi, alpha, thresholds, ws,
                                 ssmq::percentile_workspace_bytes(), stream);
}

ssmq_status ssmq_softedge_decode(const uint8_t* codes, int64_t n, float scale, int32_t log2_ratio,
                                 float* out, void* stream) {
  const char* fn = "ssmq_softedge_decode";
  Range nvtx_range(fn);
  REQUIRE(n >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  REQUIRE(log2_ratio >= 0 && log2_ratio <= 8, SSMQ_ERR_INVALID_ARG,
          "%s: log2_ratio must be in [0, 8]", fn);
  if (n > 0) REQUIRE(codes && out, SSMQ_ERR_INVALID_ARG, "%s: NULL tensor", fn);
  REQUIRE(aligned16(codes) && aligned16(out), SSMQ_ERR_ALIGNMENT, "%s: 16-byte alignment", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_softedge_decode(codes, n, scale, log2_ratio, out,
                                             (cudaStream_t)stream),
                fn);
}

ssmq_status ssmq_conv_silu_quantize(const ssmq_conv_args* a, void* stream) {
  const char* fn = "ssmq_conv_silu_quantize";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  REQUIRE(a->batch >= 0 && a->seqlen >= 0 && a->dim >= 0, SSMQ_ERR_INVALID_ARG,
          "%s: negative size", fn);
  REQUIRE(a->width >= 1 && a->width <= 4, SSMQ_ERR_INVALID_ARG, "%s: width %d not in 1..4", fn,
          (int)a->width);
  REQUIRE(a->out_format == SSMQ_X_INT8_GROUP || a->out_format == SSMQ_X_SOFTEDGE,
          SSMQ_ERR_INVALID_ARG, "%s: out_format must be INT8_GROUP or SOFTEDGE", fn);
  if (a->out_format == SSMQ_X_INT8_GROUP) {
    REQUIRE(a->x_group && a->x_scale && a->n_x_groups >= 1, SSMQ_ERR_INVALID_ARG,
            "%s: x_group, x_scale and n_x_groups >= 1 required", fn);
  } else {
    REQUIRE(a->se_lo <= a->se_hi, SSMQ_ERR_INVALID_ARG, "%s: se_lo > se_hi", fn);
    REQUIRE(a->se_log2_ratio >= 0 && a->se_log2_ratio <= 8, SSMQ_ERR_INVALID_ARG,
            "%s: se_log2_ratio must be in [0, 8]", fn);
  }
  const int64_t n = a->batch * a->dim * a->seqlen;
  const int64_t ns = a->batch * a->dim * (a->width - 1);
  if (n > 0) REQUIRE(a->x && a->weight && a->codes, SSMQ_ERR_INVALID_ARG, "%s: NULL tensor", fn);
  if (a->x_prev_out && a->x_prev && ns > 0) {
    const uintptr_t p0 = (uintptr_t)a->x_prev, p1 = (uintptr_t)a->x_prev_out;
    const uintptr_t nb = (uintptr_t)ns * sizeof(uint16_t);
    REQUIRE(p0 + nb <= p1 || p1 + nb <= p0, SSMQ_ERR_INVALID_ARG,
            "%s: x_prev_out overlaps x_prev", fn);
  }
  if (a->x_prev_out && ns > 0 && a->seqlen > 0)
    REQUIRE(a->x != nullptr, SSMQ_ERR_INVALID_ARG, "%s: x is NULL", fn);
  REQUIRE(aligned16(a->x) && aligned16(a->codes) && aligned16(a->u), SSMQ_ERR_ALIGNMENT,
          "%s: x, codes and u must be 16-byte aligned", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_conv_silu_quantize(*a, (cudaStream_t)stream), fn);
}

ssmq_status ssmq_selective_scan_w8(const ssmq_scan_args* a, void* stream) {
  const char* fn = "ssmq_selective_scan_w8";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  REQUIRE(a->batch >= 0 && a->seqlen >= 0 && a->dim >= 0, SSMQ_ERR_INVALID_ARG,
          "%s: negative size", fn);
  REQUIRE(a->ngroups >= 1 && a->dim % a->ngroups == 0, SSMQ_ERR_INVALID_ARG,
          "%s: dim must be a multiple of ngroups >= 1", fn);
  REQUIRE(a->dstate == 4 || a->dstate == 8 || a->dstate == 16 || a->dstate == 32 ||
              a->dstate == 64,
          SSMQ_ERR_UNSUPPORTED, "%s: dstate %lld not in {4, 8, 16, 32, 64}", fn,
          (long long)a->dstate);
  REQUIRE(a->state_group_size >= 1 && a->dstate % a->state_group_size == 0,
          SSMQ_ERR_INVALID_ARG, "%s: dstate must be a multiple of state_group_size", fn);
  if (a->batch == 0 || a->dim == 0) return SSMQ_OK;
  REQUIRE(aligned16(a->x) && aligned16(a->dt) && aligned16(a->z) && aligned16(a->B) &&
              aligned16(a->C) && aligned16(a->y) && aligned16(a->h0) && aligned16(a->h_final) &&
              aligned16(a->A) && aligned16(a->dec_final),
          SSMQ_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  REQUIRE(a->batch <= 65535, SSMQ_ERR_UNSUPPORTED, "%s: batch > 65535", fn);
  if (a->seqlen > 0) {
    // an empty sequence reads no token tensor (they may be NULL); the final
    // state is then the initial state
    const ssmq_status xs = check_x(a->x_format, a->x, a->x_group, a->x_scale, a->n_x_groups,
                                   a->se_log2_ratio, fn, true);
    if (xs != SSMQ_OK) return xs;
    REQUIRE(a->x_format != SSMQ_X_F16_SOFTEDGE || a->se_lo <= a->se_hi, SSMQ_ERR_INVALID_ARG,
            "%s: se_lo must not exceed se_hi (as ssmq_softedge_encode)", fn);
    REQUIRE(a->dt && a->A && a->B && a->C && a->B_scale && a->C_scale && (a->y || a->y_q),
            SSMQ_ERR_INVALID_ARG,
            "%s: a required tensor (dt, A, B, C, B_scale, C_scale, y or y_q) is NULL", fn);
    const ssmq_status ys = check_yq(a->y_q, a->y_group, a->y_scale, a->n_y_groups, fn);
    if (ys != SSMQ_OK) return ys;
    if (ssmq_scan_time_segments(a) > 1) {
      const size_t need = ssmq_scan_workspace_size(a);
      REQUIRE(a->workspace && a->workspace_bytes >= need, SSMQ_ERR_INVALID_ARG,
              "%s: %d time segments need a workspace of %zu bytes", fn,
              (int)ssmq_scan_time_segments(a), need);
      REQUIRE(aligned16(a->workspace), SSMQ_ERR_ALIGNMENT,
              "%s: workspace must be 16-byte aligned", fn);
    }
  }
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_selective_scan(*a, (cudaStream_t)stream), fn);
}

ssmq_status ssmq_selective_scan_carry_in(const ssmq_scan_args* a, const float* h_carry,
                                         void* stream) {
  const char* fn = "ssmq_selective_scan_carry_in";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  REQUIRE(a->batch >= 0 && a->seqlen >= 0 && a->dim >= 0, SSMQ_ERR_INVALID_ARG,
          "%s: negative size", fn);
  REQUIRE(a->ngroups >= 1 && a->dim % a->ngroups == 0, SSMQ_ERR_INVALID_ARG,
          "%s: dim must be a multiple of ngroups >= 1", fn);
  REQUIRE(a->dstate == 4 || a->dstate == 8 || a->dstate == 16 || a->dstate == 32 ||
              a->dstate == 64,
          SSMQ_ERR_UNSUPPORTED, "%s: dstate %lld not in {4, 8, 16, 32, 64}", fn,
          (long long)a->dstate);
  REQUIRE(a->state_group_size >= 1 && a->dstate % a->state_group_size == 0,
          SSMQ_ERR_INVALID_ARG, "%s: dstate must be a multiple of state_group_size", fn);
  if (a->batch == 0 || a->dim == 0) return SSMQ_OK;
  REQUIRE(h_carry != nullptr, SSMQ_ERR_INVALID_ARG, "%s: h_carry is NULL", fn);
  if (a->seqlen > 0)
    REQUIRE(a->y && a->dt && a->A && a->C && a->C_scale, SSMQ_ERR_INVALID_ARG,
            "%s: a required tensor (y, dt, A, C, C_scale) is NULL", fn);
  REQUIRE(aligned16(a->dt) && aligned16(a->z) && aligned16(a->C) && aligned16(a->y) &&
              aligned16(a->h_final) && aligned16(a->A) && aligned16(h_carry),
          SSMQ_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_selective_scan_carry_in(*a, h_carry, (cudaStream_t)stream), fn);
}

int32_t ssmq_scan_time_segments(const ssmq_scan_args* a) {
  if (!a) return 0;
  int64_t seg_len = 0;
  return (int32_t)ssmq::scan_time_segments(*a, &seg_len);
}

size_t ssmq_scan_workspace_size(const ssmq_scan_args* a) {
  if (!a) return 0;
  const int64_t k = ssmq_scan_time_segments(a);
  if (k <= 1 || a->batch <= 0 || a->dim <= 0 || a->dstate <= 0) return 0;
  return (size_t)k * (size_t)a->batch * (size_t)a->dim * (size_t)a->dstate * sizeof(float);
}

size_t ssmq_ssd_workspace_size(const ssmq_ssd_args* a) {
  if (!a) return 0;
  return ssmq::ssd_workspace_bytes(*a);
}

namespace {

// validation shared by the SSD scan and its carry-in; `batch` or `nheads` 0
// returns SSMQ_OK with *skip set (nothing to launch)
ssmq_status check_ssd(const ssmq_ssd_args* a, void* workspace, size_t ws_bytes, const char* fn,
                      bool* skip) {
  *skip = false;
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  REQUIRE(a->batch >= 0 && a->seqlen >= 0 && a->nheads >= 0, SSMQ_ERR_INVALID_ARG,
          "%s: negative size", fn);
  REQUIRE(a->ngroups >= 1 && a->nheads % a->ngroups == 0, SSMQ_ERR_INVALID_ARG,
          "%s: nheads must be a multiple of ngroups >= 1", fn);
  REQUIRE(a->headdim == 64 && a->dstate == 128, SSMQ_ERR_UNSUPPORTED,
          "%s: the SSD kernel runs headdim 64, dstate 128", fn);
  REQUIRE(a->chunk == 64 || a->chunk == 128 || a->chunk == 256, SSMQ_ERR_UNSUPPORTED,
          "%s: chunk must be 64, 128 or 256", fn);
  REQUIRE(a->state_group_size >= 1 && a->dstate % a->state_group_size == 0,
          SSMQ_ERR_INVALID_ARG, "%s: dstate must be a multiple of state_group_size", fn);
  REQUIRE(a->max_segments >= 0, SSMQ_ERR_INVALID_ARG, "%s: max_segments must be >= 0", fn);
  if (a->batch == 0 || a->nheads == 0) {
    *skip = true;
    return SSMQ_OK;
  }
  if (a->seqlen == 0) {  // only the state passes through (h0 or zero to h_final)
    REQUIRE(aligned16(a->h0) && aligned16(a->h_final), SSMQ_ERR_ALIGNMENT,
            "%s: tensors must be 16-byte aligned", fn);
    return SSMQ_OK;
  }
  const ssmq_status xs = check_x(a->x_format, a->x, a->x_group, a->x_scale, a->n_x_groups,
                                 a->se_log2_ratio, fn);
  if (xs != SSMQ_OK) return xs;
  REQUIRE(a->dt && a->A && a->B && a->C && a->B_scale && a->C_scale && (a->y || a->y_q),
          SSMQ_ERR_INVALID_ARG,
          "%s: a required tensor (dt, A, B, C, B_scale, C_scale, y or y_q) is NULL", fn);
  REQUIRE(aligned16(a->x) && aligned16(a->dt) && aligned16(a->z) && aligned16(a->B) &&
              aligned16(a->C) && aligned16(a->y) && aligned16(a->h0) && aligned16(a->h_final),
          SSMQ_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  const ssmq_status ys = check_yq(a->y_q, a->y_group, a->y_scale, a->n_y_groups, fn);
  if (ys != SSMQ_OK) return ys;
  const size_t need = ssmq::ssd_workspace_bytes(*a);
  REQUIRE(need == 0 || (workspace && ws_bytes >= need), SSMQ_ERR_INVALID_ARG,
          "%s: workspace of %zu bytes required (got %zu)", fn, need, ws_bytes);
  REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, SSMQ_ERR_ALIGNMENT,
          "%s: workspace must be 256-byte aligned", fn);
  return SSMQ_OK;
}

}  // namespace

ssmq_status ssmq_ssd_chunk_scan_w8(const ssmq_ssd_args* a, void* workspace, size_t ws_bytes,
                                   void* stream) {
  const char* fn = "ssmq_ssd_chunk_scan_w8";
  Range nvtx_range(fn);
  bool skip;
  CHECK(check_ssd(a, workspace, ws_bytes, fn, &skip));
  if (skip) return SSMQ_OK;
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_ssd(*a, workspace, (cudaStream_t)stream), fn);
}

ssmq_status ssmq_ssd_carry_in(const ssmq_ssd_args* a, const float* h_carry, void* workspace,
                              size_t ws_bytes, void* stream) {
  const char* fn = "ssmq_ssd_carry_in";
  Range nvtx_range(fn);
  bool skip;
  CHECK(check_ssd(a, workspace, ws_bytes, fn, &skip));
  if (skip) return SSMQ_OK;
  REQUIRE((a->y != nullptr || a->seqlen == 0) && a->y_q == nullptr, SSMQ_ERR_INVALID_ARG,
          "%s: needs the binary16 y (and no int8 y)", fn);
  REQUIRE(h_carry != nullptr, SSMQ_ERR_INVALID_ARG, "%s: h_carry is NULL", fn);
  REQUIRE(aligned16(h_carry), SSMQ_ERR_ALIGNMENT, "%s: h_carry must be 16-byte aligned", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_ssd_carry_in(*a, h_carry, workspace, (cudaStream_t)stream), fn);
}

ssmq_status ssmq_state_chain(const float* h_end, const float* dec, int32_t n_parts,
                             int64_t units, int64_t elems, float* h_out, void* stream) {
  const char* fn = "ssmq_state_chain";
  Range nvtx_range(fn);
  REQUIRE(n_parts >= 1, SSMQ_ERR_INVALID_ARG, "%s: n_parts must be >= 1", fn);
  REQUIRE(units >= 0 && elems >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  if (units == 0 || elems == 0) return SSMQ_OK;
  REQUIRE(h_end && dec && h_out, SSMQ_ERR_INVALID_ARG, "%s: NULL tensor", fn);
  REQUIRE(units <= INT64_MAX / elems / n_parts, SSMQ_ERR_INVALID_ARG, "%s: size overflow", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_state_chain(h_end, dec, n_parts, units, elems, nullptr, h_out,
                                         (cudaStream_t)stream),
                fn);
}

ssmq_status ssmq_state_update_w8(const ssmq_decode_args* a, void* stream) {
  const char* fn = "ssmq_state_update_w8";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  REQUIRE(a->batch >= 0 && a->nheads >= 0 && a->headdim >= 0, SSMQ_ERR_INVALID_ARG,
          "%s: negative size", fn);
  REQUIRE(a->ngroups >= 1 && a->nheads % a->ngroups == 0, SSMQ_ERR_INVALID_ARG,
          "%s: nheads must be a multiple of ngroups >= 1", fn);
  REQUIRE(a->dstate == 16 || a->dstate == 32 || a->dstate == 64 || a->dstate == 128,
          SSMQ_ERR_UNSUPPORTED, "%s: dstate %lld not in {16, 32, 64, 128}", fn,
          (long long)a->dstate);
  REQUIRE(a->state_group_size >= 1 && a->dstate % a->state_group_size == 0,
          SSMQ_ERR_INVALID_ARG, "%s: dstate must be a multiple of state_group_size", fn);
  if (a->batch == 0 || a->nheads == 0 || a->headdim == 0) return SSMQ_OK;
  const ssmq_status xs = check_x(a->x_format, a->x, a->x_group, a->x_scale, a->n_x_groups,
                                 a->se_log2_ratio, fn);
  if (xs != SSMQ_OK) return xs;
  REQUIRE(a->dt && a->A && a->B && a->C && a->B_scale && a->C_scale && a->state && a->y,
          SSMQ_ERR_INVALID_ARG, "%s: a required tensor is NULL", fn);
  REQUIRE(aligned16(a->state) && aligned16(a->B) && aligned16(a->C), SSMQ_ERR_ALIGNMENT,
          "%s: state, B and C must be 16-byte aligned", fn);
  REQUIRE(a->batch * a->nheads <= 0x7fffffff, SSMQ_ERR_UNSUPPORTED, "%s: too many heads", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_state_update(*a, (cudaStream_t)stream), fn);
}

ssmq_status ssmq_selective_state_update_w8(const ssmq_m1_decode_args* a, void* stream) {
  const char* fn = "ssmq_selective_state_update_w8";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  REQUIRE(a->batch >= 0 && a->dim >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  REQUIRE(a->ngroups >= 1 && a->dim % a->ngroups == 0, SSMQ_ERR_INVALID_ARG,
          "%s: dim must be a multiple of ngroups >= 1", fn);
  REQUIRE(a->dstate == 4 || a->dstate == 8 || a->dstate == 16 || a->dstate == 32 ||
              a->dstate == 64 || a->dstate == 128,
          SSMQ_ERR_UNSUPPORTED, "%s: dstate %lld not in {4, 8, 16, 32, 64, 128}", fn,
          (long long)a->dstate);
  REQUIRE(a->state_group_size >= 1 && a->dstate % a->state_group_size == 0,
          SSMQ_ERR_INVALID_ARG, "%s: dstate must be a multiple of state_group_size", fn);
  if (a->batch == 0 || a->dim == 0) return SSMQ_OK;
  const ssmq_status xs = check_x(a->x_format, a->x, a->x_group, a->x_scale, a->n_x_groups,
                                 a->se_log2_ratio, fn);
  if (xs != SSMQ_OK) return xs;
  REQUIRE(a->dt && a->A && a->B && a->C && a->B_scale && a->C_scale && a->state && a->y,
          SSMQ_ERR_INVALID_ARG, "%s: a required tensor is NULL", fn);
  REQUIRE(aligned16(a->state) && aligned16(a->A) && aligned16(a->B) && aligned16(a->C),
          SSMQ_ERR_ALIGNMENT, "%s: state, A, B and C must be 16-byte aligned", fn);
  REQUIRE(a->batch * a->dim * (a->dstate / 4) <= 0x7fffffffLL * 256, SSMQ_ERR_UNSUPPORTED,
          "%s: too many channels", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_m1_state_update(*a, (cudaStream_t)stream), fn);
}

}  // extern "C"

// ---- strided-row operators -----------------------------------------------------
namespace {

int elem_size(int32_t dtype) { return dtype == SSMQ_F32 ? 4 : 2; }
bool is_dtype(int32_t dtype) {
  return dtype == SSMQ_F32 || dtype == SSMQ_F16 || dtype == SSMQ_BF16;
}

// A (batch, rows, width) tensor of contiguous rows, as bytes.
struct Region {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty without a tensor
  int64_t bs = 0, rs = 0, width = 0;  // strides and row length in bytes
  bool any() const { return hi > lo; }
};

// Strides and alignment of a tensor's rows.  Outputs may not overlap themselves.
ssmq_status check_rows(const void* p, int64_t b, int64_t L, int64_t d, int64_t bs, int64_t rs,
                       int e, bool out, const char* name, const char* fn, Region* r) {
  *r = Region();
  if (!p) return SSMQ_OK;
  REQUIRE(reinterpret_cast<uintptr_t>(p) % (uintptr_t)e == 0, SSMQ_ERR_ALIGNMENT,
          "%s: %s is not on a %d-byte element", fn, name, e);
  if (b == 0 || L == 0 || d == 0) return SSMQ_OK;
  REQUIRE(L == 1 || rs >= d, SSMQ_ERR_INVALID_ARG, "%s: %s: row stride %lld below the row's %lld",
          fn, name, (long long)rs, (long long)d);
  REQUIRE(b == 1 || bs >= 0, SSMQ_ERR_INVALID_ARG, "%s: %s: negative batch stride", fn, name);
  const __int128 rows = (L > 1 ? (__int128)(L - 1) * rs : 0) + d;
  const __int128 all = (b > 1 ? (__int128)(b - 1) * bs : 0) + rows;
  REQUIRE(all < ((__int128)1 << 59), SSMQ_ERR_INVALID_ARG, "%s: %s: size overflow", fn, name);
  // sequence after sequence, or row after row with the sequences interleaved
  REQUIRE(!out || b == 1 || bs >= rows || (bs >= d && (__int128)(b - 1) * bs + d <= rs),
          SSMQ_ERR_INVALID_ARG, "%s: %s: batch stride %lld makes sequences overlap", fn, name,
          (long long)bs);
  r->lo = reinterpret_cast<uintptr_t>(p);
  r->hi = r->lo + (uintptr_t)all * e;
  r->bs = b > 1 ? bs * e : 0;
  r->rs = L > 1 ? rs * e : 0;
  r->width = d * e;
  return SSMQ_OK;
}
Region dense(const void* p, int64_t bytes) {
  Region r;
  if (p && bytes > 0) {
    r.lo = reinterpret_cast<uintptr_t>(p);
    r.hi = r.lo + (uintptr_t)bytes;
    r.width = bytes;
  }
  return r;
}
bool same(const Region& a, const Region& b) {
  return a.lo == b.lo && a.hi == b.hi && a.bs == b.bs && a.rs == b.rs;
}
// Whether two tensors share a byte, as far as ranges and strides tell: column
// slices of one tensor (equal strides, disjoint columns) do not.
bool overlap(const Region& a, const Region& b) {
  if (!a.any() || !b.any() || a.hi <= b.lo || b.hi <= a.lo) return false;
  if (a.rs == b.rs && a.bs == b.bs) {
    // every row of both starts a multiple of `unit` behind the first
    const int64_t less = a.rs < a.bs ? a.rs : a.bs, more = a.rs < a.bs ? a.bs : a.rs;
    const int64_t unit = less > 0 ? (more % less == 0 ? less : 0) : more;
    if (unit > 0) {
      const bool ab = a.lo < b.lo;
      const int64_t off = (int64_t)((ab ? b.lo - a.lo : a.lo - b.lo) % (uintptr_t)unit);
      if (off >= (ab ? a.width : b.width) && off + (ab ? b.width : a.width) <= unit) return false;
    }
  }
  return true;
}
struct Named {
  const char* name;
  Region r;
};
// Every output against the inputs and the other outputs; an output may be
// exactly one of the inputs flagged in `may`.
ssmq_status check_overlaps(const Named* in, const bool* may, int n_in, const Named* out, int n_out,
                           const char* fn) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      REQUIRE(!overlap(out[i].r, in[j].r) || (may[j] && same(out[i].r, in[j].r)),
              SSMQ_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out[i].name, in[j].name);
    for (int j = 0; j < i; ++j)
      REQUIRE(!overlap(out[i].r, out[j].r), SSMQ_ERR_INVALID_ARG, "%s: %s overlaps %s", fn,
              out[i].name, out[j].name);
  }
  return SSMQ_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

ssmq_status check_gated_sizes(int64_t b, int64_t L, int64_t d, int32_t dtype, const char* fn) {
  REQUIRE(is_dtype(dtype), SSMQ_ERR_INVALID_ARG, "%s: bad dtype %d", fn, (int)dtype);
  REQUIRE(b >= 0 && L >= 0 && d >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  REQUIRE(b < ((int64_t)1 << 31) && d < ((int64_t)1 << 31) && L < ((int64_t)1 << 31) &&
              b * ((d + 15) / 16) <= ((int64_t)1 << 27),
          SSMQ_ERR_UNSUPPORTED, "%s: too many steps or channels", fn);
  return SSMQ_OK;
}

}  // namespace

extern "C" {

ssmq_status ssmq_rms_norm_quantize(const ssmq_norm_args* a, void* stream) {
  const char* fn = "ssmq_rms_norm_quantize";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  REQUIRE(is_dtype(a->dtype), SSMQ_ERR_INVALID_ARG, "%s: bad dtype %d", fn, (int)a->dtype);
  REQUIRE(a->tokens >= 0 && a->dim >= 1, SSMQ_ERR_INVALID_ARG,
          "%s: need tokens >= 0 and dim >= 1", fn);
  REQUIRE(a->dim <= 32768 && a->tokens <= 0x7fffffff, SSMQ_ERR_UNSUPPORTED,
          "%s: dim > 32768 or tokens > 2^31 - 1", fn);
  REQUIRE(a->eps >= 0.0f, SSMQ_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  REQUIRE((a->codes != nullptr) == (a->scales != nullptr), SSMQ_ERR_INVALID_ARG,
          "%s: codes and scales come together", fn);
  if (a->tokens == 0) return SSMQ_OK;
  REQUIRE(a->x && (a->codes || a->y), SSMQ_ERR_INVALID_ARG, "%s: x, or every output, is NULL", fn);
  REQUIRE(aligned4(a->weight) && aligned4(a->scales) && aligned4(a->status), SSMQ_ERR_ALIGNMENT,
          "%s: weight, scales and status must be 4-byte aligned", fn);
  const int e = elem_size(a->dtype);
  Named in[3] = {{"x", {}}, {"residual", {}}, {"weight", dense(a->weight, 4 * a->dim)}};
  Named out[4] = {{"residual_out", {}}, {"y", {}}, {"codes", {}},
                  {"scales", dense(a->scales, 4 * a->tokens)}};
  CHECK(check_rows(a->x, 1, a->tokens, a->dim, 0, a->x_stride, e, false, "x", fn, &in[0].r));
  CHECK(check_rows(a->residual, 1, a->tokens, a->dim, 0, a->residual_stride, e, false, "residual",
                   fn, &in[1].r));
  CHECK(check_rows(a->residual_out, 1, a->tokens, a->dim, 0, a->residual_out_stride, e, true,
                   "residual_out", fn, &out[0].r));
  CHECK(check_rows(a->y, 1, a->tokens, a->dim, 0, a->y_stride, e, true, "y", fn, &out[1].r));
  CHECK(check_rows(a->codes, 1, a->tokens, a->dim, 0, a->codes_stride, 1, true, "codes", fn,
                   &out[2].r));
  const bool in_place[3] = {true, true, false}, never[3] = {false, false, false};
  CHECK(check_overlaps(in, in_place, 3, out, 1, fn));
  CHECK(check_overlaps(in, never, 3, out + 1, 3, fn));
  for (int i = 1; i < 4; ++i)
    REQUIRE(!overlap(out[0].r, out[i].r), SSMQ_ERR_INVALID_ARG, "%s: residual_out overlaps %s", fn,
            out[i].name);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_rms_norm_quantize(*a, (cudaStream_t)stream), fn);
}

size_t ssmq_int8_linear_workspace_size(const ssmq_linear_args* a) {
  return a ? ssmq::int8_linear_workspace_bytes(*a) : 0;
}

ssmq_status ssmq_int8_linear(const ssmq_linear_args* a, void* workspace, size_t ws_bytes,
                             void* stream) {
  const char* fn = "ssmq_int8_linear";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  REQUIRE(is_dtype(a->dtype), SSMQ_ERR_INVALID_ARG, "%s: bad dtype %d", fn, (int)a->dtype);
  const int64_t M = a->tokens, N = a->out_features, K = a->in_features;
  REQUIRE(M >= 0 && N >= 0 && K >= 0, SSMQ_ERR_INVALID_ARG, "%s: negative size", fn);
  REQUIRE(K <= 131071, SSMQ_ERR_UNSUPPORTED,
          "%s: in_features > 131071 (32-bit sums could overflow)", fn);
  REQUIRE(M <= 0x7fffffff && N <= 0x7fffffff, SSMQ_ERR_UNSUPPORTED,
          "%s: more than 2^31 - 1 tokens or channels", fn);
  if (M == 0 || N == 0) return SSMQ_OK;
  REQUIRE(a->x_scale && a->w_scale && a->y && (K == 0 || (a->x && a->w)), SSMQ_ERR_INVALID_ARG,
          "%s: a required tensor is NULL", fn);
  REQUIRE(aligned4(a->x_scale) && aligned4(a->w_scale) && aligned4(a->bias) &&
              aligned4(a->status),
          SSMQ_ERR_ALIGNMENT, "%s: scales, bias and status must be 4-byte aligned", fn);
  Named in[5] = {{"x", {}}, {"w", {}}, {"x_scale", dense(a->x_scale, 4 * M)},
                 {"w_scale", dense(a->w_scale, 4 * N)}, {"bias", dense(a->bias, 4 * N)}};
  Named out[1] = {{"y", {}}};
  CHECK(check_rows(a->x, 1, M, K, 0, a->x_stride, 1, false, "x", fn, &in[0].r));
  CHECK(check_rows(a->w, 1, N, K, 0, a->w_stride, 1, false, "w", fn, &in[1].r));
  CHECK(check_rows(a->y, 1, M, N, 0, a->y_stride, elem_size(a->dtype), true, "y", fn, &out[0].r));
  REQUIRE(a->x_stride < ((int64_t)1 << 40) && a->w_stride < ((int64_t)1 << 40),
          SSMQ_ERR_UNSUPPORTED, "%s: row stride of 2^40 bytes or more", fn);
  const bool never[5] = {};
  CHECK(check_overlaps(in, never, 5, out, 1, fn));
  const size_t need = ssmq::int8_linear_workspace_bytes(*a);
  if (need) {
    REQUIRE(workspace && ws_bytes >= need, SSMQ_ERR_INVALID_ARG,
            "%s: workspace of %zu bytes required (got %zu)", fn, need, ws_bytes);
    REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 255u) == 0, SSMQ_ERR_ALIGNMENT,
            "%s: workspace must be 256-byte aligned", fn);
    const Named room[1] = {{"the workspace", dense(workspace, (int64_t)need)}};
    CHECK(check_overlaps(in, never, 5, room, 1, fn));
    REQUIRE(!overlap(room[0].r, out[0].r), SSMQ_ERR_INVALID_ARG, "%s: y overlaps the workspace",
            fn);
  }
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_int8_linear(*a, workspace, (cudaStream_t)stream), fn);
}

int32_t ssmq_gated_scan_state_steps(void) { return ssmq::kGatedStateSteps; }

ssmq_status ssmq_gated_scan(const ssmq_gated_args* a, void* stream) {
  const char* fn = "ssmq_gated_scan";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const int64_t b = a->batch, L = a->seqlen, d = a->dim;
  CHECK(check_gated_sizes(b, L, d, a->dtype, fn));
  if (b == 0 || d == 0) return SSMQ_OK;
  REQUIRE(L == 0 || (a->v.p && a->g.p && a->y.p), SSMQ_ERR_INVALID_ARG, "%s: v, g or y is NULL",
          fn);
  REQUIRE(aligned4(a->h0) && aligned4(a->h_final) && aligned4(a->states) && aligned4(a->lengths) &&
              aligned4(a->status),
          SSMQ_ERR_ALIGNMENT, "%s: h0, h_final, states, lengths and status must be 4-byte aligned",
          fn);
  const int e = elem_size(a->dtype);
  const int64_t saved = (L + ssmq::kGatedStateSteps - 1) / ssmq::kGatedStateSteps;
  Named in[5] = {{"z", {}}, {"v", {}}, {"g", {}}, {"h0", dense(a->h0, 4 * b * d)},
                 {"lengths", dense(a->lengths, 4 * b)}};
  Named out[3] = {{"y", {}}, {"h_final", dense(a->h_final, 4 * b * d)},
                  {"states", dense(a->states, 4 * b * saved * d)}};
  const ssmq_rows* rows[4] = {&a->z, &a->v, &a->g, &a->y};
  for (int i = 0; i < 4; ++i)
    CHECK(check_rows(rows[i]->p, b, L, d, rows[i]->batch_stride, rows[i]->row_stride, e, i == 3,
                     i < 3 ? in[i].name : "y", fn, i < 3 ? &in[i].r : &out[0].r));
  const bool may_y[5] = {true, false, false, false, false};
  const bool may_h[5] = {false, false, false, true, false}, never[5] = {};
  CHECK(check_overlaps(in, may_y, 5, out, 1, fn));
  CHECK(check_overlaps(in, may_h, 5, out + 1, 1, fn));
  CHECK(check_overlaps(in, never, 5, out + 2, 1, fn));
  REQUIRE(!overlap(out[1].r, out[2].r), SSMQ_ERR_INVALID_ARG, "%s: states overlaps h_final", fn);
  for (int i = 1; i < 3; ++i)
    REQUIRE(!overlap(out[0].r, out[i].r), SSMQ_ERR_INVALID_ARG, "%s: y overlaps %s", fn,
            out[i].name);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_gated_scan(*a, (cudaStream_t)stream), fn);
}

ssmq_status ssmq_gated_scan_backward(const ssmq_gated_grad_args* a, void* stream) {
  const char* fn = "ssmq_gated_scan_backward";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const int64_t b = a->batch, L = a->seqlen, d = a->dim;
  CHECK(check_gated_sizes(b, L, d, a->dtype, fn));
  if (b == 0 || d == 0) return SSMQ_OK;
  REQUIRE(L == 0 || (a->v.p && a->g.p && a->dy.p && a->states && a->dv.p && a->dg.p),
          SSMQ_ERR_INVALID_ARG, "%s: v, g, dy, states, dv or dg is NULL", fn);
  REQUIRE(L == 0 || (a->z.p != nullptr) == (a->dz.p != nullptr), SSMQ_ERR_INVALID_ARG,
          "%s: z and dz come together", fn);
  REQUIRE(aligned4(a->states) && aligned4(a->dh_final) && aligned4(a->dh0) &&
              aligned4(a->lengths) && aligned4(a->status),
          SSMQ_ERR_ALIGNMENT,
          "%s: states, dh_final, dh0, lengths and status must be 4-byte aligned", fn);
  const int e = elem_size(a->dtype);
  const int64_t saved = (L + ssmq::kGatedStateSteps - 1) / ssmq::kGatedStateSteps;
  Named in[7] = {{"v", {}}, {"g", {}}, {"z", {}}, {"dy", {}},
                 {"states", dense(a->states, 4 * b * saved * d)},
                 {"dh_final", dense(a->dh_final, 4 * b * d)},
                 {"lengths", dense(a->lengths, 4 * b)}};
  Named out[4] = {{"dv", {}}, {"dg", {}}, {"dz", {}}, {"dh0", dense(a->dh0, 4 * b * d)}};
  const ssmq_rows* rows[7] = {&a->v, &a->g, &a->z, &a->dy, &a->dv, &a->dg, &a->dz};
  for (int i = 0; i < 7; ++i)
    CHECK(check_rows(rows[i]->p, b, L, d, rows[i]->batch_stride, rows[i]->row_stride, e, i >= 4,
                     i < 4 ? in[i].name : out[i - 4].name, fn, i < 4 ? &in[i].r : &out[i - 4].r));
  const bool may[7] = {true, true, true, true, false, false, false};
  const bool may_dh[7] = {false, false, false, false, false, true, false};
  CHECK(check_overlaps(in, may, 7, out, 3, fn));
  CHECK(check_overlaps(in, may_dh, 7, out + 3, 1, fn));
  for (int i = 0; i < 3; ++i)
    REQUIRE(!overlap(out[i].r, out[3].r), SSMQ_ERR_INVALID_ARG, "%s: dh0 overlaps %s", fn,
            out[i].name);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_gated_scan_backward(*a, (cudaStream_t)stream), fn);
}

ssmq_status ssmq_gated_update(const ssmq_gated_args* a, void* stream) {
  const char* fn = "ssmq_gated_update";
  Range nvtx_range(fn);
  REQUIRE(a != nullptr, SSMQ_ERR_INVALID_ARG, "%s: args is NULL", fn);
  const int64_t b = a->batch, d = a->dim;
  CHECK(check_gated_sizes(b, a->seqlen, d, a->dtype, fn));
  REQUIRE(a->seqlen == 1, SSMQ_ERR_INVALID_ARG, "%s: seqlen must be 1", fn);
  REQUIRE(!a->states && !a->lengths, SSMQ_ERR_INVALID_ARG,
          "%s: states and lengths must be NULL", fn);
  if (b == 0 || d == 0) return SSMQ_OK;
  REQUIRE(a->v.p && a->g.p && a->y.p && a->h_final, SSMQ_ERR_INVALID_ARG,
          "%s: v, g, y or the state (h_final) is NULL", fn);
  REQUIRE(aligned4(a->h_final), SSMQ_ERR_ALIGNMENT, "%s: the state must be 4-byte aligned", fn);
  const int e = elem_size(a->dtype);
  Named in[3] = {{"z", {}}, {"v", {}}, {"g", {}}};
  Named out[2] = {{"y", {}}, {"the state", dense(a->h_final, 4 * b * d)}};
  const ssmq_rows* rows[4] = {&a->z, &a->v, &a->g, &a->y};
  // (the sequences are the rows of one batch)
  for (int i = 0; i < 4; ++i)
    CHECK(check_rows(rows[i]->p, b, 1, d, rows[i]->batch_stride, d, e, i == 3,
                     i < 3 ? in[i].name : "y", fn, i < 3 ? &in[i].r : &out[0].r));
  for (Region* r : {&in[0].r, &in[1].r, &in[2].r, &out[0].r}) {
    r->rs = r->bs;
    r->bs = 0;
  }
  const bool may[3] = {true, false, false}, never[3] = {false, false, false};
  CHECK(check_overlaps(in, may, 3, out, 1, fn));
  CHECK(check_overlaps(in, never, 3, out + 1, 1, fn));
  REQUIRE(!overlap(out[0].r, out[1].r), SSMQ_ERR_INVALID_ARG, "%s: y overlaps the state", fn);
  if (injected(fn)) return fail(SSMQ_ERR_CUDA, "%s: injected launch failure", fn);
  return finish(ssmq::launch_gated_update(*a, (cudaStream_t)stream), fn);
}

}  // extern "C"
