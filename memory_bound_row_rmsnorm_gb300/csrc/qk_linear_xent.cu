// qk_linear_xent.cu -- cross-entropy of a linear layer's logits, forward and
// backward, without the logits in memory.
//
//   logits = h w^T;  lse = log sum exp(logits);  loss = lse - logits[t] + z lse^2
//   g = dloss ((1 + 2 z lse) exp(logits - lse) - onehot(t));  dh = g w;  dw = g^T h
//
// The vocabulary is walked in pieces: a piece's logits (fp32) are formed in the
// workspace, folded into each row's running (maximum, sum) pair or turned into
// g, and overwritten by the next piece's.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/qk.h"
#include "qk_host.h"
#include "qk_kernels.cuh"  // xent_mean_kernel

namespace qk {
namespace {

constexpr int64_t kMaxDim = INT32_MAX;
constexpr int64_t kPieceBytes = int64_t(256) << 20;  // a piece's logits in the workspace

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

struct XentRow {  // what an epilogue needs of a row
  float lse, g, zf;
  int32_t target;  // -1: none
};

// ---------------------------------------------------------------------------
// C[i,j] (+)= sum_k A(i,k) B(j,k) in fp32: 64 x 64 tiles, 16 of k at a time in
// shared memory, 4 x 4 results a thread.  Element (i,k) of A is at
// i * a_row + k * a_col, of B at j * b_row + k * b_col.
// ---------------------------------------------------------------------------
struct ProductArgs {
  const void* a;
  const void* b;
  void* c;
  int64_t a_row, a_col, b_row, b_col, c_row;
  int64_t rows, cols, depth;
  int32_t add;        // add to C
  const float* scale; // factor on the result (device), may be null
};

template <typename TA, typename TB, typename TC>
__global__ void __launch_bounds__(256) product_kernel(const ProductArgs p) {
  __shared__ float as[16][65], bs[16][65];
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t i0 = int64_t(blockIdx.y) * 64, j0 = int64_t(blockIdx.x) * 64;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.depth; k0 += 16) {
    for (int e = tid; e < 64 * 16; e += 256) {
      const int kk = e & 15, rr = e >> 4;
      const int64_t k = k0 + kk;
      as[kk][rr] = i0 + rr < p.rows && k < p.depth
                       ? Vec16<TA>::load1(static_cast<const TA*>(p.a) + (i0 + rr) * p.a_row + k * p.a_col) : 0.f;
      bs[kk][rr] = j0 + rr < p.cols && k < p.depth
                       ? Vec16<TB>::load1(static_cast<const TB*>(p.b) + (j0 + rr) * p.b_row + k * p.b_col) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(as[kk][ty + 16 * u], bs[kk][tx + 16 * v], acc[u][v]);
    __syncthreads();
  }
  const float f = p.scale != nullptr ? *p.scale : 1.f;
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
      if (i >= p.rows || j >= p.cols) continue;
      TC* c = static_cast<TC*>(p.c) + i * p.c_row + j;
      const float r = acc[u][v] * f;
      Vec16<TC>::store1(c, p.add ? Vec16<TC>::load1(c) + r : r);
    }
}

template <typename TA, typename TB, typename TC>
qk_status product(const ProductArgs& p, void* stream) {
  const dim3 grid(unsigned((p.cols + 63) / 64), unsigned((p.rows + 63) / 64));
  return launch_pdl(product_kernel<TA, TB, TC>, grid, 256, 0, stream, p);
}

// Folds a piece's logits into each row's (maximum, sum) pair; one CTA a row.
__global__ void __launch_bounds__(256) fold_kernel(const float* logits, int64_t ld, int64_t v0, int64_t width,
                                                   const int64_t* targets, float2* state, float* at_target) {
  __shared__ float2 red[8];
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t row = blockIdx.x;
  const float* x = logits + row * ld;
  float m = kNegInf, s = 0.f;
  for (int64_t j = threadIdx.x; j < width; j += 256) m = fmaxf(m, x[j]);
  for (int64_t j = threadIdx.x; j < width; j += 256)
    if (x[j] != kNegInf) s += exp2_approx((x[j] - m) * kLog2e);
  group_ms<32>(m, s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x != 0) return;
  float2 t = v0 > 0 ? state[row] : make_float2(kNegInf, 0.f);
  for (int i = 0; i < 8; ++i) {
    const float mn = fmaxf(t.x, red[i].x);
    t.y = (t.x == kNegInf ? t.y : t.y * exp2_approx((t.x - mn) * kLog2e)) +
          (red[i].x == kNegInf ? red[i].y : red[i].y * exp2_approx((red[i].x - mn) * kLog2e));
    t.x = mn;
  }
  state[row] = t;
  const int64_t c = targets[row] - v0;
  if (c >= 0 && c < width) at_target[row] = x[c];
}

__global__ void __launch_bounds__(256) loss_kernel(const float2* state, const float* at_target,
                                                   const int64_t* targets, int64_t M, int64_t V, int has_ignore,
                                                   int64_t ignore_index, float z, float* loss, float* lse) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t row = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (row >= M) return;
  const float l = state[row].x + logf(state[row].y);
  const int64_t t = targets[row];
  if (lse != nullptr) lse[row] = l;
  loss[row] = has_ignore && t == ignore_index ? 0.f
              : t >= 0 && t < V               ? fmaf(z * l, l, l - at_target[row])
                                              : __int_as_float(0x7fc00000);
}

// A piece's logits into its g, in place.
__global__ void __launch_bounds__(256) grad_kernel(float* logits, int64_t ld, int64_t v0, int64_t width, int64_t V,
                                                   const int64_t* targets, const float* lse, const float* dloss,
                                                   int has_ignore, int64_t ignore_index, float z) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t row = blockIdx.x;
  float* x = logits + row * ld;
  const int64_t t = targets[row];
  const bool ignored = has_ignore && t == ignore_index;
  const float l = lse[row], zf = fmaf(2.f * z, l, 1.f);
  const float g = t >= 0 && t < V ? (dloss != nullptr ? dloss[row] : 1.f) : __int_as_float(0x7fc00000);
  for (int64_t j = threadIdx.x; j < width; j += 256) {
    const float p = exp2_approx((x[j] - l) * kLog2e) * zf - (v0 + j == t ? 1.f : 0.f);
    x[j] = ignored ? 0.f : g * p;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) round_kernel(const float* in, T* out, int64_t n) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) Vec16<T>::store1(out + i, in[i]);
}

struct Layout {
  int64_t piece;  // vocabulary rows of one piece
  int64_t logits, state, at_target, dh, total;  // byte offsets
};
Layout layout(int64_t M, int64_t V, int64_t K) {
  Layout l;
  l.piece = std::min(V, std::max<int64_t>(64, kPieceBytes / 4 / M / 64 * 64));
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  l.logits = take(M * l.piece * 4);
  l.state = take(M * 8);
  l.at_target = take(M * 4);
  l.dh = take(M * K * 4);
  l.total = at;
  return l;
}

qk_status check_linear(int dtype, int64_t M, int64_t V, int64_t K) {
  if (dtype != QK_F32 && dtype != QK_BF16) return QK_ERR_INVALID_ARG;
  if (M < 0 || V <= 0 || K <= 0) return QK_ERR_INVALID_ARG;
  if (M > kMaxDim || V > kMaxDim || K > kMaxDim) return QK_ERR_UNSUPPORTED;
  return QK_OK;
}

struct Call {
  const void* h;
  const void* w;
  const int64_t* targets;
  int64_t M, V, K;
  int has_ignore;
  int64_t ignore;
  float z;
  char* ws;
  void* stream;
};

template <typename T>
qk_status logits_piece(const Call& c, const Layout& l, int64_t v0, int64_t width) {
  ProductArgs p = {};
  p.a = c.h, p.a_row = c.K, p.a_col = 1;
  p.b = static_cast<const T*>(c.w) + v0 * c.K, p.b_row = c.K, p.b_col = 1;
  p.c = c.ws + l.logits, p.c_row = l.piece;
  p.rows = c.M, p.cols = width, p.depth = c.K;
  return product<T, T, float>(p, c.stream);
}

template <typename T>
qk_status forward(const Call& c, float* loss, float* lse) {
  const Layout l = layout(c.M, c.V, c.K);
  float2* state = reinterpret_cast<float2*>(c.ws + l.state);
  float* at = reinterpret_cast<float*>(c.ws + l.at_target);
  for (int64_t v0 = 0; v0 < c.V; v0 += l.piece) {
    const int64_t width = std::min(l.piece, c.V - v0);
    qk_status st = logits_piece<T>(c, l, v0, width);
    if (st == QK_OK)
      st = launch_pdl(fold_kernel, dim3(unsigned(c.M)), 256, 0, c.stream,
                      reinterpret_cast<const float*>(c.ws + l.logits), l.piece, v0, width, c.targets, state, at);
    if (st != QK_OK) return st;
  }
  return launch_pdl(loss_kernel, dim3(unsigned((c.M + 255) / 256)), 256, 0, c.stream, state, at, c.targets, c.M,
                    c.V, c.has_ignore, c.ignore, c.z, loss, lse);
}

template <typename T>
qk_status backward(const Call& c, const float* lse, const float* dloss, void* dh, void* dw) {
  const Layout l = layout(c.M, c.V, c.K);
  float* g = reinterpret_cast<float*>(c.ws + l.logits);
  float* sum = reinterpret_cast<float*>(c.ws + l.dh);
  for (int64_t v0 = 0; v0 < c.V; v0 += l.piece) {
    const int64_t width = std::min(l.piece, c.V - v0);
    qk_status st = logits_piece<T>(c, l, v0, width);
    if (st == QK_OK)
      st = launch_pdl(grad_kernel, dim3(unsigned(c.M)), 256, 0, c.stream, g, l.piece, v0, width, c.V, c.targets,
                      lse, dloss, c.has_ignore, c.ignore, c.z);
    ProductArgs p = {};
    p.a = g, p.a_row = l.piece, p.a_col = 1;
    p.b = static_cast<const T*>(c.w) + v0 * c.K, p.b_row = 1, p.b_col = c.K;
    p.c = sum, p.c_row = c.K;
    p.rows = c.M, p.cols = c.K, p.depth = width;
    p.add = v0 > 0;
    if (st == QK_OK && dh != nullptr) st = product<float, T, float>(p, c.stream);
    p.a_row = 1, p.a_col = l.piece;
    p.b = c.h;
    p.c = static_cast<T*>(dw) + v0 * c.K;
    p.rows = width, p.depth = c.M;
    p.add = 0;
    if (st == QK_OK && dw != nullptr) st = product<float, T, T>(p, c.stream);
    if (st != QK_OK) return st;
  }
  if (dh == nullptr) return QK_OK;
  return launch_pdl(round_kernel<T>, dim3(unsigned((c.M * c.K + 255) / 256)), 256, 0, c.stream,
                    reinterpret_cast<const float*>(sum), static_cast<T*>(dh), c.M * c.K);
}

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

qk_status qk_linear_xent_fwd_workspace_size(int64_t M, int64_t V, int64_t K, qk_dtype dtype, size_t* bytes) {
  if (bytes == nullptr) return QK_ERR_INVALID_ARG;
  *bytes = 0;
  const qk_status st = check_linear(dtype, M, V, K);
  if (st != QK_OK || M == 0) return st;
  *bytes = size_t(layout(M, V, K).total);
  return QK_OK;
}

qk_status qk_linear_xent_bwd_workspace_size(int64_t M, int64_t V, int64_t K, qk_dtype dtype, size_t* bytes) {
  return qk_linear_xent_fwd_workspace_size(M, V, K, dtype, bytes);
}

qk_status qk_linear_xent_fwd(const void* h, const void* w, const int64_t* targets, float* loss, float* lse,
                             float* mean_loss, void* workspace, size_t workspace_bytes, int64_t M, int64_t V,
                             int64_t K, qk_dtype dtype, const qk_xent_options* options, void* stream) {
  const int has_ignore = options != nullptr && options->has_ignore_index != 0;
  const int64_t ignore = has_ignore ? options->ignore_index : 0;
  const float z = options != nullptr ? options->z_loss : 0.f;
  qk_status st = check_linear(dtype, M, V, K);
  if (st != QK_OK) return st;
  if (!std::isfinite(z)) return QK_ERR_INVALID_ARG;
  if (!aligned_to(mean_loss, 4)) return QK_ERR_MISALIGNED;
  if (M > 0) {
    if (h == nullptr || w == nullptr || targets == nullptr || loss == nullptr || workspace == nullptr)
      return QK_ERR_INVALID_ARG;
    const size_t es = size_t(elem_size(dtype));
    if (!aligned_to(h, es) || !aligned_to(w, es) || !aligned_to(targets, 8) || !aligned_to(loss, 4) ||
        !aligned_to(lse, 4) || !aligned_to(workspace, 256))
      return QK_ERR_MISALIGNED;
    size_t need = 0;
    st = qk_linear_xent_fwd_workspace_size(M, V, K, dtype, &need);
    if (st != QK_OK) return st;
    if (workspace_bytes < need) return QK_ERR_INVALID_ARG;
    const struct {
      const void* p;
      int64_t n;
    } in[] = {{h, M * K * int64_t(es)}, {w, V * K * int64_t(es)}, {targets, M * 8}},
      out[] = {{loss, M * 4}, {lse, M * 4}, {mean_loss, 4}, {workspace, int64_t(need)}};
    for (int i = 0; i < 4; ++i) {
      for (const auto& b : in)
        if (overlap(out[i].p, out[i].n, b.p, b.n)) return QK_ERR_INVALID_ARG;
      for (int k = i + 1; k < 4; ++k)
        if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return QK_ERR_INVALID_ARG;
    }
  }
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  const Call c = {h, w, targets, M, V, K, has_ignore, ignore, z, static_cast<char*>(workspace), stream};
  if (M > 0) st = dtype == QK_F32 ? forward<float>(c, loss, lse) : forward<__nv_bfloat16>(c, loss, lse);
  if (st != QK_OK || mean_loss == nullptr) return st;
  return launch_pdl(xent_mean_kernel<0>, dim3(1), 1024, 0, stream, loss, targets, M, has_ignore, ignore,
                    mean_loss);
}

qk_status qk_linear_xent_bwd(const void* h, const void* w, const int64_t* targets, const float* lse,
                             const float* dloss, void* dh, void* dw, void* workspace, size_t workspace_bytes,
                             int64_t M, int64_t V, int64_t K, qk_dtype dtype, const qk_xent_options* options,
                             void* stream) {
  const int has_ignore = options != nullptr && options->has_ignore_index != 0;
  const int64_t ignore = has_ignore ? options->ignore_index : 0;
  const float z = options != nullptr ? options->z_loss : 0.f;
  qk_status st = check_linear(dtype, M, V, K);
  if (st != QK_OK) return st;
  if (!std::isfinite(z)) return QK_ERR_INVALID_ARG;
  const size_t es = size_t(elem_size(dtype));
  const int64_t wb = V * K * int64_t(es);
  if (!aligned_to(dw, es)) return QK_ERR_MISALIGNED;
  if (M > 0) {
    if (h == nullptr || w == nullptr || targets == nullptr || lse == nullptr || workspace == nullptr)
      return QK_ERR_INVALID_ARG;
    if (!aligned_to(h, es) || !aligned_to(w, es) || !aligned_to(dh, es) || !aligned_to(targets, 8) ||
        !aligned_to(lse, 4) || !aligned_to(dloss, 4) || !aligned_to(workspace, 256))
      return QK_ERR_MISALIGNED;
    size_t need = 0;
    st = qk_linear_xent_bwd_workspace_size(M, V, K, dtype, &need);
    if (st != QK_OK) return st;
    if (workspace_bytes < need) return QK_ERR_INVALID_ARG;
    const struct {
      const void* p;
      int64_t n;
    } in[] = {{h, M * K * int64_t(es)}, {w, wb}, {targets, M * 8}, {lse, M * 4}, {dloss, M * 4}},
      out[] = {{dh, M * K * int64_t(es)}, {dw, wb}, {workspace, int64_t(need)}};
    for (int i = 0; i < 3; ++i) {
      for (const auto& b : in)
        if (overlap(out[i].p, out[i].n, b.p, b.n)) return QK_ERR_INVALID_ARG;
      for (int k = i + 1; k < 3; ++k)
        if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return QK_ERR_INVALID_ARG;
    }
  }
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  if (M == 0) {  // a sum over no rows
    if (dw == nullptr ||
        cudaMemsetAsync(dw, 0, size_t(wb), static_cast<cudaStream_t>(stream)) == cudaSuccess)
      return QK_OK;
    cudaGetLastError();
    return QK_ERR_LAUNCH;
  }
  const Call c = {h, w, targets, M, V, K, has_ignore, ignore, z, static_cast<char*>(workspace), stream};
  return dtype == QK_F32 ? backward<float>(c, lse, dloss, dh, dw)
                         : backward<__nv_bfloat16>(c, lse, dloss, dh, dw);
}

}  // extern "C"
