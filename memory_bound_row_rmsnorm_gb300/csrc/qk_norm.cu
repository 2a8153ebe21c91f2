// qk_norm.cu -- C ABI of RMSNorm with the residual's addition: argument checks,
// plans, launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <map>
#include <mutex>
#include <tuple>

#include "../../include/qk.h"
#include "qk_bwd_kernels.cuh"  // dw_reduce_kernel
#include "qk_host.h"
#include "qk_norm_kernels.cuh"
#include "qk_norm_ring.cuh"

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

// How a call runs: a ring kernel, or the any-row kernel (func == nullptr).
struct NormPlan {
  const void* func = nullptr;
  int threads = 0, slots = 0, smem = 0;
  uint32_t slot_bytes = 0;
  int64_t items = 0, grid = 0;
};

std::mutex g_norm_mu;
std::map<std::tuple<int, const void*, int>, int> g_norm_occ;  // (device, kernel, smem) -> CTAs an SM

// Resident CTAs an SM; opts the kernel into the device's shared memory first.
qk_status norm_occupancy(const CurrentDevice& d, const void* func, int threads, int smem, int* out) try {
  std::lock_guard<std::mutex> lock(g_norm_mu);
  const auto key = std::make_tuple(d.index, func, smem);
  const auto it = g_norm_occ.find(key);
  if (it != g_norm_occ.end()) {
    *out = it->second;
    return QK_OK;
  }
  int n = 0;
  if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem_optin - kNormStaticSmem) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, func, threads, size_t(smem)) != cudaSuccess) {
    cudaGetLastError();
    return QK_ERR_LAUNCH;
  }
  *out = g_norm_occ[key] = n;
  return QK_OK;
} catch (...) {  // no exception leaves a C entry point
  return QK_ERR_LAUNCH;
}

NormTable shapes_of(int op, int dtype, bool vec) {
  switch (op * 2 + (dtype == QK_BF16)) {
    case 2 * kAddNorm: return norm_shapes_add_f32(vec);
    case 2 * kAddNorm + 1: return norm_shapes_add_bf16(vec);
    case 2 * kNormQuant: return norm_shapes_quant_f32(vec);
    case 2 * kNormQuant + 1: return norm_shapes_quant_bf16(vec);
    case 2 * kAddNormBwd: return norm_shapes_bwd_f32(vec);
    default: return norm_shapes_bwd_bf16(vec);
  }
}

// The first shape that holds the row, a ring of one or two items, a grid of
// every resident CTA.
qk_status plan_norm(const CurrentDevice& d, int op, int dtype, int64_t M, int64_t N, bool vec, int inputs,
                    NormPlan* p) {
  *p = NormPlan{};
  const int es = elem_size(dtype);
  const int64_t units = vec ? N * es / 16 : N;
  const NormTable t = shapes_of(op, dtype, vec);
  const NormShape* s = nullptr;
  for (int i = 0; i < t.count && s == nullptr; ++i)
    if (units <= t.shapes[i].units) s = &t.shapes[i];
  if (s == nullptr) {
    p->grid = any_grid(d, M);
    return QK_OK;
  }
  const int R = s->threads / s->row_threads;
  p->func = s->func;
  p->threads = s->threads;
  p->items = (M + R - 1) / R;
  p->slot_bytes = uint32_t((int64_t(R) * N * es + (vec ? 0 : 31) + 127) / 128 * 128);
  // Ring slots, from runs of 1 to 4 at nine shapes.  Two by default (three and
  // four cost the backward 3 to 6 % at 16384 x 4096 and 8192 x 8192 in bf16, and
  // change the forward by 1 %); one for the 8-bit output of rows of up to 1024
  // vectors in launches of at least 8 items a CTA, whose registers and
  // arithmetic want more CTAs an SM (16384 x 4096 bf16, a scale a row: 82 us
  // with two, 75 with one; 4096 x 4096: 18.7 and 19.6); three for the backward
  // of aligned rows in launches of fewer than 8 items a CTA, where fewer CTAs
  // leave fewer partial rows of dw to sum (2049 x 2048 fp32: 18.9 us, 14.6).
  auto with_slots = [&](int slots, int* smem, int* occ) {
    const int64_t bytes = kSmemHeader + int64_t(slots) * inputs * p->slot_bytes;
    *smem = int(bytes);
    *occ = 0;
    return bytes > d.smem_optin - kNormStaticSmem ? QK_OK : norm_occupancy(d, s->func, s->threads, *smem, occ);
  };
  int best = 0;
  for (int slots = 2; slots >= 1; --slots) {
    int smem, occ;
    const qk_status st = with_slots(slots, &smem, &occ);
    if (st != QK_OK) return st;
    if (occ == 0) continue;
    const bool one = op == kNormQuant && units <= 1024 && p->items >= 8 * int64_t(occ) * d.sms;
    if (best == 0 || one) best = occ, p->slots = slots, p->smem = smem;
    if (!one) break;
  }
  if (op == kAddNormBwd && vec && p->slots == 2 && p->items < 8 * int64_t(best) * d.sms) {
    int smem, occ;
    const qk_status st = with_slots(3, &smem, &occ);
    if (st != QK_OK) return st;
    if (occ > 0) best = occ, p->slots = 3, p->smem = smem;
  }
  if (best == 0) return QK_ERR_UNSUPPORTED;
  p->grid = std::min<int64_t>(p->items, int64_t(best) * d.sms);
  return QK_OK;
}

// The plan of a call, kept per thread for the last shape of each operator and type.
qk_status norm_plan(const CurrentDevice& d, int op, int dtype, int64_t M, int64_t N, bool vec, int inputs,
                    NormPlan* out) {
  struct Cached {
    int dev = -1, inputs = 0;
    int64_t M = -1, N = -1;
    NormPlan plan;
  };
  thread_local Cached cache[3][2][2];
  Cached& c = cache[op][dtype == QK_BF16][vec];
  if (!(c.dev == d.index && c.M == M && c.N == N && c.inputs == inputs)) {
    NormPlan p;
    const qk_status st = plan_norm(d, op, dtype, M, N, vec, inputs, &p);
    if (st != QK_OK) return st;
    c.dev = d.index, c.M = M, c.N = N, c.inputs = inputs, c.plan = p;
  }
  *out = c.plan;
  return QK_OK;
}

// Whether the rows of all these pointers are whole 16-byte vectors (the 8-bit
// output's: whole groups of the 4 or 8 bytes that belong to one).
bool whole_vectors(int dtype, int64_t N, std::initializer_list<const void*> ptrs) {
  if (N * int64_t(elem_size(dtype)) % 16 != 0) return false;
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  return true;
}

template <int OP>
qk_status run_norm(const CurrentDevice& d, int dtype, NormArgs& a, bool vec, void* stream) {
  NormPlan p;
  const int inputs = 1 + (a.r != nullptr) + (a.r2 != nullptr);
  const qk_status st = norm_plan(d, OP, dtype, a.M, a.N, vec, inputs, &p);
  if (st != QK_OK) return st;
  a.inv_n = float(1.0 / double(a.N));
  a.timeout_ns = kWaitTimeoutNs;
  a.status = d.status;
  if (p.func == nullptr) return launch_any<OP>(d, dtype, a, stream);
  a.slots = p.slots;
  a.slot_bytes = p.slot_bytes;
  a.num_items = p.items;
  return launch_pdl(reinterpret_cast<void (*)(NormArgs)>(const_cast<void*>(p.func)), dim3(unsigned(p.grid)),
                    p.threads, size_t(p.smem), stream, a);
}

// Rows of dw partials of a backward launch: the most that either way of it
// takes (kept per thread for the last shape).
qk_status bwd_partial_rows(const CurrentDevice& d, int dtype, int64_t M, int64_t N, int64_t* rows) {
  thread_local struct {
    int dev = -1, dtype = 0;
    int64_t M = 0, N = 0, rows = 0;
  } last;
  if (last.dev == d.index && last.dtype == dtype && last.M == M && last.N == N) {
    *rows = last.rows;
    return QK_OK;
  }
  *rows = 0;
  for (int inputs = 2; inputs <= 3; ++inputs)
    for (const bool vec : {false, true}) {
      if (vec && N * int64_t(elem_size(dtype)) % 16 != 0) continue;
      NormPlan p;
      const qk_status st = plan_norm(d, kAddNormBwd, dtype, M, N, vec, inputs, &p);
      if (st != QK_OK) return st;
      *rows = std::max(*rows, p.grid);
    }
  last.dev = d.index, last.dtype = dtype, last.M = M, last.N = N, last.rows = *rows;
  return QK_OK;
}

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
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  return run_norm<kAddNorm>(d, dtype, a, whole_vectors(dtype, N, {x, residual, w, y, h}), stream);
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
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  const bool vec = whole_vectors(dtype, N, {x, residual, w, h}) && aligned_to(q, 16 / es);
  return run_norm<kNormQuant>(d, dtype, a, vec, stream);
}

qk_status qk_add_rmsnorm_bwd_workspace_size(int64_t M, int64_t N, qk_dtype dtype, size_t* bytes) {
  if (bytes == nullptr) return QK_ERR_INVALID_ARG;
  *bytes = 0;
  qk_status st = check_rows(dtype, M, N);
  if (st != QK_OK || M == 0) return st;
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  int64_t rows = 0;
  st = bwd_partial_rows(d, dtype, M, N, &rows);
  *bytes = size_t(rows) * size_t(N) * 4;
  return st;
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
  const bool vec = whole_vectors(dtype, N, {h, w, dy, dh, dx});
  NormPlan p;
  st = norm_plan(d, kAddNormBwd, dtype, M, N, vec, dh != nullptr ? 3 : 2, &p);
  if (st != QK_OK) return st;
  const int64_t rows = p.grid;
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
  st = run_norm<kAddNormBwd>(d, dtype, a, vec, stream);
  if (st != QK_OK) return st;
  const float* part = a.dw_partial;
  return launch_pdl(dw_reduce_kernel<0>, dim3(unsigned((N + 31) / 32)), kDwReduceThreads, 0, stream, part, dw,
                    rows, N);
}

}  // extern "C"
