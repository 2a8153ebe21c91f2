// qk_norm.cu -- C ABI of RMSNorm with the residual's addition: argument checks,
// plans, launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/qk.h"
#include "qk_bwd_kernels.cuh"  // dw_reduce_kernel
#include "qk_host.h"
#include "qk_norm_kernels.cuh"

namespace qk {
namespace {

// M and N of a row operator (any row length is served).
qk_status check_rows(int dtype, int64_t M, int64_t N) {
  if (dtype != QK_F32 && dtype != QK_BF16) return QK_ERR_INVALID_ARG;
  if (M < 0 || N <= 0) return QK_ERR_INVALID_ARG;
  if (M > 0 && N > INT64_MAX / 16 / M) return QK_ERR_INVALID_ARG;  // byte offsets fit int64
  return QK_OK;
}

// CTAs of the any-row kernel: four of its 256 threads an SM keep enough loads
// in flight, and bound the backward's partial rows.
int64_t any_grid(const CurrentDevice& d, int64_t M) { return std::min<int64_t>(M, 4 * int64_t(d.sms)); }

template <int OP>
qk_status launch_any(const CurrentDevice& d, int dtype, const NormArgs& a, void* stream) {
  const dim3 grid(unsigned(any_grid(d, a.M)));
  return dtype == QK_F32 ? launch_pdl(norm_any_kernel<OP, float>, grid, kNormAnyThreads, 0, stream, a)
                         : launch_pdl(norm_any_kernel<OP, __nv_bfloat16>, grid, kNormAnyThreads, 0, stream, a);
}

template <int OP>
qk_status run_norm(int dtype, NormArgs& a, void* stream) {
  CurrentDevice d;
  const qk_status st = current_device(&d);
  if (st != QK_OK) return st;
  a.inv_n = float(1.0 / double(a.N));
  a.timeout_ns = kWaitTimeoutNs;
  a.status = d.status;
  return launch_any<OP>(d, dtype, a, stream);
}

// Rows of dw partials of a backward launch.
int64_t bwd_partial_rows(const CurrentDevice& d, int64_t M) { return any_grid(d, M); }

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

qk_status qk_add_rmsnorm_fwd(const void* x, const void* residual, const void* w, void* y, void* h,
                             float* rstd, int64_t M, int64_t N, float eps, qk_dtype dtype, void* stream) {
  qk_status st = check_rows(dtype, M, N);
  if (st != QK_OK) return st;
  if (!(std::isfinite(eps) && eps >= 0.f)) return QK_ERR_INVALID_ARG;
  if (M == 0) return QK_OK;
  if (x == nullptr || residual == nullptr || w == nullptr || y == nullptr || h == nullptr)
    return QK_ERR_INVALID_ARG;
  const size_t es = size_t(elem_size(dtype));
  for (const void* p : {x, residual, w, static_cast<const void*>(y), static_cast<const void*>(h)})
    if (!aligned_to(p, es)) return QK_ERR_MISALIGNED;
  if (!aligned_to(rstd, 4)) return QK_ERR_MISALIGNED;
  const int64_t bytes = M * N * int64_t(es), wb = N * int64_t(es), rb = M * 4;
  for (const void* o : {static_cast<const void*>(y), static_cast<const void*>(h)}) {
    if ((o != x && overlap(o, bytes, x, bytes)) || (o != residual && overlap(o, bytes, residual, bytes)) ||
        overlap(o, bytes, w, wb) || overlap(o, bytes, rstd, rb))
      return QK_ERR_INVALID_ARG;
  }
  if (overlap(y, bytes, h, bytes) || overlap(rstd, rb, x, bytes) || overlap(rstd, rb, residual, bytes) ||
      overlap(rstd, rb, w, wb))
    return QK_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = x;
  a.r = residual;
  a.w = w;
  a.y = y;
  a.h = h;
  a.rstd = rstd;
  a.M = M;
  a.N = N;
  a.eps = eps;
  return run_norm<kAddNorm>(dtype, a, stream);
}

qk_status qk_rmsnorm_quant_fwd(const void* x, const void* residual, const void* w, void* q, float* scale,
                               void* h, float* rstd, int64_t M, int64_t N, float eps, int64_t group,
                               qk_dtype dtype, qk_qtype qtype, void* stream) {
  qk_status st = check_rows(dtype, M, N);
  if (st != QK_OK) return st;
  if (!(std::isfinite(eps) && eps >= 0.f)) return QK_ERR_INVALID_ARG;
  if (group != 0 && group != 32 && group != 64 && group != 128) return QK_ERR_INVALID_ARG;
  if (qtype != QK_E4M3 && qtype != QK_INT8) return QK_ERR_INVALID_ARG;
  if (M == 0) return QK_OK;
  if (x == nullptr || w == nullptr || q == nullptr || scale == nullptr) return QK_ERR_INVALID_ARG;
  if (residual == nullptr && h != nullptr) return QK_ERR_INVALID_ARG;
  const size_t es = size_t(elem_size(dtype));
  for (const void* p : {x, residual, w, static_cast<const void*>(h)})
    if (!aligned_to(p, es)) return QK_ERR_MISALIGNED;
  if (!aligned_to(scale, 4) || !aligned_to(rstd, 4)) return QK_ERR_MISALIGNED;
  const int64_t groups = group == 0 ? 1 : (N + group - 1) / group;
  const int64_t bytes = M * N * int64_t(es), wb = N * int64_t(es), rb = M * 4, qb = M * N, sb = M * groups * 4;
  const struct {
    const void* p;
    int64_t n;
  } out[] = {{q, qb}, {scale, sb}, {rstd, rb}, {h, bytes}};
  for (int i = 0; i < 4; ++i) {
    if ((out[i].p != x || i < 3) && overlap(out[i].p, out[i].n, x, bytes)) return QK_ERR_INVALID_ARG;
    if ((out[i].p != residual || i < 3) && overlap(out[i].p, out[i].n, residual, bytes))
      return QK_ERR_INVALID_ARG;
    if (overlap(out[i].p, out[i].n, w, wb)) return QK_ERR_INVALID_ARG;
    for (int k = i + 1; k < 4; ++k)
      if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return QK_ERR_INVALID_ARG;
  }
  NormArgs a = {};
  a.x = x;
  a.r = residual;
  a.w = w;
  a.y = q;
  a.h = h;
  a.scale = scale;
  a.rstd = rstd;
  a.M = M;
  a.N = N;
  a.eps = eps;
  a.group = int32_t(group);
  a.groups = groups;
  a.qtype = qtype;
  return run_norm<kNormQuant>(dtype, a, stream);
}

qk_status qk_add_rmsnorm_bwd_workspace_size(int64_t M, int64_t N, qk_dtype dtype, size_t* bytes) {
  if (bytes == nullptr) return QK_ERR_INVALID_ARG;
  *bytes = 0;
  qk_status st = check_rows(dtype, M, N);
  if (st != QK_OK || M == 0) return st;
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  *bytes = size_t(bwd_partial_rows(d, M)) * size_t(N) * 4;
  return QK_OK;
}

qk_status qk_add_rmsnorm_bwd(const void* h, const void* w, const float* rstd, const void* dy, const void* dh,
                             void* dx, float* dw, void* workspace, size_t workspace_bytes, int64_t M,
                             int64_t N, qk_dtype dtype, void* stream) {
  qk_status st = check_rows(dtype, M, N);
  if (st != QK_OK) return st;
  if (dw == nullptr) return QK_ERR_INVALID_ARG;
  if (!aligned_to(dw, 4)) return QK_ERR_MISALIGNED;
  if (M > 0) {
    if (h == nullptr || w == nullptr || rstd == nullptr || dy == nullptr || dx == nullptr ||
        workspace == nullptr)
      return QK_ERR_INVALID_ARG;
    const size_t es = size_t(elem_size(dtype));
    for (const void* p : {h, w, dy, dh, static_cast<const void*>(dx)})
      if (!aligned_to(p, es)) return QK_ERR_MISALIGNED;
    if (!aligned_to(rstd, 4) || !aligned_to(workspace, 16)) return QK_ERR_MISALIGNED;
    const int64_t bytes = M * N * int64_t(es), wb = N * int64_t(es), rb = M * 4;
    const int64_t wsb = int64_t(std::min<size_t>(workspace_bytes, size_t(INT64_MAX)));
    for (const void* in : {h, dy, dh})
      if ((dx != in && overlap(dx, bytes, in, bytes)) || overlap(dw, N * 4, in, bytes) ||
          overlap(workspace, wsb, in, bytes))
        return QK_ERR_INVALID_ARG;
    if (overlap(dx, bytes, w, wb) || overlap(dx, bytes, rstd, rb) || overlap(dx, bytes, dw, N * 4) ||
        overlap(dx, bytes, workspace, wsb) || overlap(dw, N * 4, w, wb) || overlap(dw, N * 4, rstd, rb) ||
        overlap(workspace, wsb, dw, N * 4) || overlap(workspace, wsb, w, wb) ||
        overlap(workspace, wsb, rstd, rb))
      return QK_ERR_INVALID_ARG;
  }
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  if (M == 0) {  // a sum over no rows
    if (cudaMemsetAsync(dw, 0, size_t(N) * 4, static_cast<cudaStream_t>(stream)) == cudaSuccess) return QK_OK;
    cudaGetLastError();
    return QK_ERR_LAUNCH;
  }
  const int64_t rows = bwd_partial_rows(d, M);
  if (workspace_bytes < size_t(rows) * size_t(N) * 4) return QK_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = h;
  a.r = dy;
  a.r2 = dh;
  a.w = w;
  a.rstd = const_cast<float*>(rstd);  // read only
  a.y = dx;
  a.dw_partial = static_cast<float*>(workspace);
  a.M = M;
  a.N = N;
  st = run_norm<kAddNormBwd>(dtype, a, stream);
  if (st != QK_OK) return st;
  const float* part = a.dw_partial;
  return launch_pdl(dw_reduce_kernel<0>, dim3(unsigned((N + 31) / 32)), kDwReduceThreads, 0, stream, part, dw,
                    rows, N);
}

}  // extern "C"
