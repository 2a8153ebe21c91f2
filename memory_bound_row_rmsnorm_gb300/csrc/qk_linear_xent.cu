// qk_linear_xent.cu -- cross-entropy of a linear layer's logits, forward and
// backward, without the logits in memory.
//
//   logits = h w^T;  lse = log sum exp(logits);  loss = lse - logits[t] + z lse^2
//   g = dloss ((1 + 2 z lse) exp(logits - lse) - onehot(t));  dh = g w;  dw = g^T h
//
// Forward: one product whose epilogue folds each 128 columns of a row into
// a (maximum, sum of exponentials) pair, then a join of the pairs of a row.
// Backward, for one piece of the vocabulary after the other: a product whose
// epilogue turns logits into g (bf16, in the workspace), dh += g w[piece] in
// fp32, and dw[piece] = g^T h, complete at once.  A piece is as wide as keeps
// its g within kPieceBytes, so the workspace does not grow with the vocabulary.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/qk.h"
#include "qk_bwd_kernels.cuh"  // dw_reduce_kernel
#include "qk_few_tokens.cuh"
#include "qk_host.h"
#include "qk_kernels.cuh"  // xent_mean_kernel
#include "qk_product_kernel.cuh"
#include "qk_tensor_map.h"

namespace qk {
namespace {

constexpr int64_t kMaxDim = INT32_MAX - 15;  // TMA coordinates, and rows padded to 8, are 32-bit
constexpr int64_t kPieceBytes = int64_t(256) << 20;  // g of one piece
constexpr int64_t kStageCopyBytes = int64_t(256) << 20;  // copied or split weights of one piece: enough for a wave of tiles
constexpr int kPairs = 76;  // CTA pairs of a GB300
// Up to this many bf16 tokens the forward puts the vocabulary on the tile's rows and
// the tokens on its 16 to 64 columns.  With tokens on the 256 rows the tensor
// cores work through 240 empty ones at 16 tokens, 34 us at 32000 x 4096 where
// reading w takes 39 us at the copy's rate; the columns cost them nothing.
constexpr int64_t kFewTokens = 64;
constexpr int64_t kFewSmem = 200 << 10;  // h of the fp32 kernels for few tokens, in shared memory

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }

// ---------------------------------------------------------------------------
// Small kernels around the products
// ---------------------------------------------------------------------------

// Rows of T into rows of bf16 planes whose row length is a multiple of 8 (what
// TMA wants): float32 in three planes, bf16 (an unaligned tensor) copied.  A warp
// takes a row; a lane takes 8 neighbouring columns at a time where the rows are
// float32 vectors (VEC), else 2, so that a warp's loads and stores are whole
// lines.  What lies behind the last column is read by nobody.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) planes_kernel(const T* in, int64_t rows, int32_t cols, __nv_bfloat16* out,
                                                     int32_t ld, int64_t plane_stride) {
  static_assert(!VEC || sizeof(T) == 4, "16-byte loads of four floats");
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int kCols = VEC ? 8 : 2, kUnroll = VEC ? 2 : 4;
  const int lane = threadIdx.x & 31;
  for (int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); i < rows; i += int64_t(gridDim.x) * 8) {
    const T* src = in + i * cols;
    __nv_bfloat16* dst = out + i * ld;
    for (int64_t j0 = kCols * lane; j0 < cols; j0 += 32 * kCols * kUnroll) {
      T x[kUnroll][kCols];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = j0 + 32 * kCols * u;
        if constexpr (VEC) {  // cols is a multiple of 4
#pragma unroll
          for (int e = 0; e < kCols; e += 4) {
            const float4 v = j + e < cols ? *reinterpret_cast<const float4*>(src + j + e) : float4{};
            x[u][e] = v.x, x[u][e + 1] = v.y, x[u][e + 2] = v.z, x[u][e + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < kCols; ++e) x[u][e] = j + e < cols ? src[j + e] : T(0.f);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = j0 + 32 * kCols * u;
        if (j >= cols) break;  // ld is a multiple of 8: the columns stay inside the row
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<__nv_bfloat162*>(dst + j) = __nv_bfloat162{x[u][0], x[u][1]};
        } else {
          uint32_t o[3][kCols / 2];
#pragma unroll
          for (int e = 0; e < kCols; e += 2) {
            __nv_bfloat16 a[3], b[3];
            split3(x[u][e], a);
            split3(x[u][e + 1], b);
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) {
              const __nv_bfloat162 v{a[pl], b[pl]};
              o[pl][e / 2] = *reinterpret_cast<const uint32_t*>(&v);
            }
          }
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {
            __nv_bfloat16* to = dst + pl * plane_stride + j;
            if constexpr (VEC) {
              *reinterpret_cast<uint4*>(to) = make_uint4(o[pl][0], o[pl][1], o[pl][2], o[pl][3]);
            } else {
              *reinterpret_cast<uint32_t*>(to) = o[pl][0];
            }
          }
        }
      }
    }
  }
}

// A plane's rows [rows][ld_in] into [cols][ld_out], 64 x 64 elements a CTA.
__global__ void __launch_bounds__(256) transpose_kernel(const uint16_t* in, int64_t rows, int64_t cols, int64_t ld_in,
                                                        int64_t plane_in, uint16_t* out, int64_t ld_out,
                                                        int64_t plane_out) {
  __shared__ uint16_t tile[64][66];
  grid_dependency_wait();
  allow_dependent_launch();
  const int64_t r0 = int64_t(blockIdx.x) * 64, c0 = int64_t(blockIdx.y) * 64;
  in += blockIdx.z * plane_in;
  out += blockIdx.z * plane_out;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;  // two elements of a row
#pragma unroll
  for (int i = y; i < 64; i += 8) {
    const int64_t r = r0 + i, c = c0 + 2 * x;
    // ld_in is a multiple of 8 elements and so is the base: pairs are aligned
    uint32_t v = 0;
    if (r < rows && c < cols) v = *reinterpret_cast<const uint32_t*>(in + r * ld_in + c);
    tile[i][2 * x] = uint16_t(v);
    tile[i][2 * x + 1] = uint16_t(v >> 16);
  }
  __syncthreads();
#pragma unroll
  for (int i = y; i < 64; i += 8) {
    const int64_t c = c0 + i, r = r0 + 2 * x;
    if (c < cols && r < ld_out)
      *reinterpret_cast<uint32_t*>(out + c * ld_out + r) =
          uint32_t(tile[2 * x][i]) | uint32_t(tile[2 * x + 1][i]) << 16;
  }
}

// A row's (maximum, sum) of exponentials, joined from pairs in a fixed order.
struct Joined {
  float m = kNegInf, s = 0.f;
  __device__ __forceinline__ void fold(float2 b) {  // an empty (-inf) side adds its sum, 0 or NaN
    const float mn = fmaxf(m, b.x);
    s = (m == kNegInf ? s : s * exp2_approx((m - mn) * kLog2e)) +
        (b.x == kNegInf ? b.y : b.y * exp2_approx((b.x - mn) * kLog2e));
    m = mn;
  }
  // Pairs t, t + 32, ... of n, four loads in flight.
  __device__ __forceinline__ void fold_list(const float2* part, int64_t ld, int64_t row, int64_t t, int64_t n) {
    for (; t < n; t += 4 * 32) {
      float2 b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = t + k * 32 < n ? part[(t + k * 32) * ld + row] : make_float2(kNegInf, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) fold(b[k]);
    }
  }
};

struct LossArgs {
  const float2* part;
  int64_t part_ld, n;  // n pairs a row
  const float* at_target;
  const int64_t* targets;
  int64_t M, V;
  int32_t has_ignore;
  float z;
  int64_t ignore_index;
  float* loss;
  float* lse;
  float* mean;
};
__device__ __forceinline__ bool ignored(const LossArgs& a, int64_t t) { return a.has_ignore && t == a.ignore_index; }
// Writes a row's lse and loss; returns the loss.
__device__ __forceinline__ float put_loss(const LossArgs& a, int64_t row, const Joined& j) {
  const float l = j.m + logf(j.s);
  const int64_t t = a.targets[row];
  const float loss = ignored(a, t)       ? 0.f
                     : t >= 0 && t < a.V ? fmaf(a.z * l, l, l - a.at_target[row])
                                         : __int_as_float(0x7fc00000);
  if (a.lse != nullptr) a.lse[row] = l;
  a.loss[row] = loss;
  return loss;
}

// Lanes are rows and the CTA's 32 warps take every 32nd pair.
__global__ void __launch_bounds__(1024) join_kernel(const LossArgs a) {
  __shared__ float2 red[32][33];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = int64_t(blockIdx.x) * 32 + lane;
  Joined j;
  if (row < a.M) j.fold_list(a.part, a.part_ld, row, warp, a.n);
  red[warp][lane] = make_float2(j.m, j.s);
  __syncthreads();
  if (warp != 0 || row >= a.M) return;
  j = Joined{};
  for (int i = 0; i < 32; ++i) j.fold(red[i][lane]);
  put_loss(a, row, j);
}

// Few rows (at most 64), one CTA: a warp is a row, its lanes take every 32nd
// pair; the mean over the rows that count follows at once.
__global__ void __launch_bounds__(1024) join_few_kernel(const LossArgs a) {
  __shared__ float loss[64];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t row = warp; row < a.M; row += 32) {
    Joined j;
    j.fold_list(a.part, a.part_ld, row, lane, a.n);
    const float m = group_max<32>(j.m);
    j.s = group_sum<32>(j.m == kNegInf ? j.s : j.s * exp2_approx((j.m - m) * kLog2e));
    j.m = m;
    if (lane == 0) loss[row] = put_loss(a, row, j);
  }
  __syncthreads();
  if (a.mean == nullptr || threadIdx.x != 0) return;
  float sum = 0.f;
  int n = 0;
  for (int64_t row = 0; row < a.M; ++row)
    if (!ignored(a, a.targets[row])) sum += loss[row], ++n;
  *a.mean = sum / float(n);  // 0 / 0 = NaN when every row is ignored
}

// What the gradient needs of each row.  g is dloss over the largest |dloss| of
// the rows that count, which `scale` keeps for the outputs: the mean's constant
// gradient then is 1, and g's bf16 rounding does not see its size.  One CTA.
__global__ void __launch_bounds__(1024) rows_kernel(const int64_t* targets, const float* lse, const float* dloss,
                                                    int64_t M, int64_t V, int has_ignore, int64_t ignore_index,
                                                    float z, XentRow* row, float* scale) {
  __shared__ float red[32];
  grid_dependency_wait();
  allow_dependent_launch();
  auto ignored = [&](int64_t t) { return has_ignore && t == ignore_index; };
  float c = 1.f;
  if (dloss != nullptr) {
    c = 0.f;
    for (int64_t i = threadIdx.x; i < M; i += 1024)
      if (!ignored(targets[i])) c = fmaxf(c, fabsf(dloss[i]));
    c = group_max<32>(c);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = c;
    __syncthreads();
    c = group_max<32>(red[threadIdx.x & 31]);
    if (!(c > 0.f && c < __int_as_float(0x7f800000))) c = 1.f;
  }
  if (threadIdx.x == 0) *scale = c;
  for (int64_t i = threadIdx.x; i < M; i += 1024) {
    const int64_t t = targets[i];
    const bool ok = t >= 0 && t < V;
    XentRow r;
    r.lse = lse[i];
    r.g = !ok ? __int_as_float(0x7fc00000) : dloss != nullptr ? dloss[i] / c : 1.f;
    r.zf = fmaf(2.f * z, r.lse, 1.f);
    r.target = ignored(t) ? -2 : ok ? int32_t(t) : -1;
    row[i] = r;
  }
}

// dh from its fp32 sums: the splits in order, rounded once.  A thread takes 4
// columns of a row (the sums' rows are multiples of 8).
template <typename T>
__global__ void __launch_bounds__(256) finish_kernel(const float* sum, int32_t ld, int64_t split_stride, int splits,
                                                     T* out, int64_t rows, int32_t cols) {
  grid_dependency_wait();
  allow_dependent_launch();
  const uint32_t per_row = uint32_t(ld) / 4;
  for (int64_t i0 = blockIdx.x; i0 * 256 < rows * per_row; i0 += gridDim.x) {
    const int64_t unit = i0 * 256 + threadIdx.x, i = unit / per_row;
    if (i >= rows) return;
    const int32_t j = int32_t(unit - i * per_row) * 4;
    const float4* s = reinterpret_cast<const float4*>(sum + i * ld + j);
    float4 v = s[0];
    for (int k0 = 1; k0 < splits; k0 += 8) {  // eight loads in flight
      float4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < splits) x[k] = s[(k0 + k) * (split_stride / 4)];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < splits) v = make_float4(v.x + x[k].x, v.y + x[k].y, v.z + x[k].z, v.w + x[k].w);
    }
    const float f[4] = {v.x, v.y, v.z, v.w};
    T* o = out + i * cols + j;
    if (cols % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(T) - 1)) == 0) {
      if (j >= cols) continue;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(o) = make_uint2(Vec16<T>::pack2(f[0], f[1]), Vec16<T>::pack2(f[2], f[3]));
      } else {
        *reinterpret_cast<float4*>(o) = v;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < cols) Vec16<T>::store1(o + e, f[e]);
    }
  }
}

// ---------------------------------------------------------------------------
// Plans: pieces, splits, workspace
// ---------------------------------------------------------------------------
struct Layout {
  int planes;
  int64_t kp;          // row length of copied operands and of dh's sums
  int64_t piece;       // vocabulary rows of one piece, a multiple of 256 unless it is all
  int64_t ld_g;        // row length of g
  int splits, split_steps;  // k splits of dh's product
  // byte offsets
  int64_t h, w, part, at_target, row, scale, g, sum, ht, total;
  bool turned;         // dw's product reads h as [K][M]
  int few;             // tokens of the fp32 kernels for few tokens (0: the products)
  int few_grid;        // CTAs of the logits, each with a pair a token
  int few_chunk;       // k of h in their shared memory
  int few_kv;          // backward: columns of a thread
  int columns, splits_y;  // backward: threads of a CTA along k, splits of the vocabulary by CTAs
  int64_t per_split;
};

// Launches are waves of kPairs tiles; a wave takes as long as its tiles have
// steps of 64 k.
int64_t waves(int64_t tiles) { return ceil_div(tiles, kPairs); }

// Vocabulary rows of a piece, at most `most` (or 256) of them and whole tiles.
// What the last wave of a piece's two products over the vocabulary's tiles (g,
// dw) leaves idle depends on the number of tiles, and a launch costs some 10
// steps: the cheapest count by that, from half of the most on.  (8192 x 32000 x
// 4096: 63 + 62 tiles wide take 27 + 27 and 14 + 13 waves.)
int64_t choose_piece(int64_t M, int64_t V, int64_t K, int64_t most) {
  const int64_t all = ceil_div(V, kTileN), mt = ceil_div(M, kTileM), kt = ceil_div(K, kTileN);
  const int64_t top = std::max<int64_t>(1, most / kTileN);
  if (top >= all) return V;
  int64_t best = top, best_cost = INT64_MAX;
  for (int64_t w = top; w >= (top + 1) / 2; --w) {
    const int64_t full = all / w, rest = all % w;
    auto cost = [&](int64_t n) { return n == 0 ? 0 : waves(n * mt) * ceil_div(K, kStepK) + waves(n * kt) * ceil_div(M, kStepK) + 30; };
    const int64_t c = full * cost(w) + cost(rest);
    if (c < best_cost) best = w, best_cost = c;
  }
  return best * kTileN;
}

// k splits of dh's product over a piece: with few tiles (few rows, or a narrow
// model) they give every pair work, with many they even out the last wave; each
// costs a pass of fp32 sums through memory (written, and read once more).  The
// 0.27 us of a step only weigh it against those bytes: near what the tensor
// cores' nominal rate takes.  At the rate of a measured burst it is 0.33, in a
// long run under the power limit 0.37 (8192 x 32000 x 4096 forward: 53 waves of
// 64 steps in 1271 us), and a float32 step's six products take some 1.8 (4096 x
// 16384 x 1024 forward: 14 waves of 16 in 437 us, 40 of them for the planes).
int choose_splits(int64_t M, int64_t K, int64_t steps, int products) {
  const int64_t tiles = ceil_div(M, kTileM) * ceil_div(K, kTileN);
  int best = 1;
  double best_us = 1e30;
  for (int s = 1; s <= kPairs && int64_t(s) * 16 <= std::max<int64_t>(steps * products, 16); ++s) {
    const double us = double(waves(tiles * s)) * double(ceil_div(steps, s) * products) * 0.27 + (s > 1 ? s : 0) * (double(M) * double(K) * 8 / 6.0e6);
    if (us < 0.97 * best_us) best = s, best_us = us;
  }
  return best;
}

// `copied`: h and w go through the workspace (float32, or rows that TMA cannot read in place).
Layout plan_layout(bool bwd, int64_t M, int64_t V, int64_t K, int dtype, bool copied) {
  Layout l = {};
  l.planes = dtype == QK_F32 ? 3 : 1;
  l.kp = round_up(K, 8);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  };
  // Few float32 tokens: the fp32 kernels (qk_few_tokens.cuh), while g stays within a piece.
  // The backward of 17 to 32 tokens multiplies more than it moves: by the fp32
  // kernels 83 us at 8000 x 1024, 147 at 16000 x 1024, 536 at 30000 x 2048 and
  // 338 at 8000 x 4096; by the products 95, 134, 444 and 282.  (The forward: 30,
  // 49, 226 and 124 us; by the products 47, 66, 276 and 179.)
  const int mt = M <= 4 ? 4 : M <= 8 ? 8 : M <= 16 ? 16 : 32;
  const int64_t most_few = bwd && V > (int64_t(1) << 24) / K ? 16 : 32;
  if (dtype == QK_F32 && M <= most_few && V * mt * 4 <= kPieceBytes) {
    l.few = mt;
    l.few_chunk = int(std::min<int64_t>(round_up(K, 128), kFewSmem / (mt * 4) / 128 * 128));
    l.few_grid = int(std::min<int64_t>(ceil_div(V, 16 * (64 / mt > 8 ? 8 : 64 / mt)), 2 * kPairs));
    l.piece = V;
    // columns of a thread in the backward: 64 sums and 64 values of h in registers
    l.few_kv = K % 4 != 0 ? 1 : mt <= 8 ? 4 : mt == 16 ? 2 : 1;
    const int64_t threads = ceil_div(K, l.few_kv);
    l.columns = threads <= 64 ? 64 : threads <= 128 ? 128 : 256;
    if (!bwd) {
      l.part = take(int64_t(l.few_grid) * M * 8);
      l.at_target = take(M * 4);
    } else {
      // two CTAs an SM, twice over, each with at least 64 rows of the vocabulary
      const int64_t across = ceil_div(threads, l.columns);
      const int64_t y = std::max<int64_t>(1, std::min<int64_t>(8 * kPairs / across, ceil_div(V, 64)));
      l.per_split = round_up(ceil_div(V, y), 64);
      l.splits_y = int(ceil_div(V, l.per_split));
      l.splits = l.splits_y * (kFewThreads / l.columns);
      l.row = take(M * int64_t(sizeof(XentRow)));
      l.scale = take(4);
      l.g = take(V * mt * 4);
      l.sum = take(int64_t(l.splits) * M * K * 4);
    }
    l.total = at;
    return l;
  }
  int64_t most = round_up(V, 256);
  if (copied) most = std::min<int64_t>(most, kStageCopyBytes / (l.kp * 2 * l.planes));
  if (bwd) most = std::min<int64_t>(most, kPieceBytes / (M * 2 * l.planes));
  l.piece = bwd ? choose_piece(M, V, K, most) : std::min<int64_t>(V, std::max<int64_t>(kTileN, most / kTileN * kTileN));
  if (copied) {
    l.h = take(l.planes * M * l.kp * 2);
    l.w = take(l.planes * l.piece * l.kp * 2);
  }
  if (!bwd) {
    const int64_t pairs = M > kFewTokens || l.planes == 3
                              ? 2 * ceil_div(V, kTileN)
                              : 2 * std::min<int64_t>(ceil_div(V, kTileM), kPairs * ceil_div(V, l.piece));
    l.part = take(pairs * M * 8);
    l.at_target = take(M * 4);
  } else {
    // dw = g^T h reads both operands MN-major, at which the tensor cores run
    // slower than on K-major ones.  A copy of h as [K][M] makes one of them
    // K-major: 5680 -> 5363 us at 8192 x 131072 x 4096, 1509 -> 1430 at 8192 x
    // 32000 x 4096, but 66 -> 68 at 1001 x 50257 x 768, where the copy costs what
    // it gains.  And a K-major operand takes a last column tile of 32 columns
    // where an MN-major one takes 128 (2047 x 8191 x 513).
    const int64_t rest = K % kTileN;
    l.turned = (double(M) * double(V) * double(K) > 1e11 || (rest > 0 && rest <= 96)) && K <= 65535 * 64;
    if (l.turned) l.ht = take(l.planes * K * round_up(M, 8) * 2);
    l.row = take(M * int64_t(sizeof(XentRow)));
    l.scale = take(4);
    l.ld_g = round_up(l.piece, 8);
    l.g = take(l.planes * M * l.ld_g * 2);
    const int64_t steps = ceil_div(l.piece, kStepK);
    const int splits = choose_splits(M, K, steps, l.planes == 3 ? 6 : 1);
    l.split_steps = int(ceil_div(steps, splits));
    l.splits = int(ceil_div(steps, l.split_steps));
    l.sum = take(int64_t(l.splits) * M * l.kp * 4);
  }
  l.total = at;
  return l;
}

// The same, kept per thread for the last sizes of each kind.
const Layout& layout(bool bwd, int64_t M, int64_t V, int64_t K, int dtype, bool copied) {
  struct Cached {
    int64_t M = -1, V = -1, K = -1;
    Layout l;
  };
  thread_local Cached cache[2][2][2];
  Cached& c = cache[bwd][dtype == QK_BF16][copied];
  if (c.M != M || c.V != V || c.K != K) {
    c.l = plan_layout(bwd, M, V, K, dtype, copied);
    c.M = M, c.V = V, c.K = K;
  }
  return c.l;
}

qk_status check_linear(int dtype, int64_t M, int64_t V, int64_t K) {
  if (dtype != QK_F32 && dtype != QK_BF16) return QK_ERR_INVALID_ARG;
  if (M < 0 || V <= 0 || K <= 0) return QK_ERR_INVALID_ARG;
  if (M > kMaxDim || V > kMaxDim || K > kMaxDim) return QK_ERR_UNSUPPORTED;
  if (std::max(M, V) > INT64_MAX / 1024 / K) return QK_ERR_UNSUPPORTED;  // byte offsets fit int64
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
  CurrentDevice dev;
};

// ---------------------------------------------------------------------------
// Tensor maps and launches
// ---------------------------------------------------------------------------
// A bf16 operand [planes][rows][ld] of which the first `inner` columns count.
struct Operand {
  const void* base;
  int64_t inner, rows, ld, planes, plane_stride;  // elements
};

// Boxes of 64 x box_rows in 128-byte swizzle; what lies outside reads as zero.
bool make_map(CUtensorMap* map, const Operand& o, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {cuuint64_t(o.inner), cuuint64_t(o.rows), cuuint64_t(o.planes)};
  const cuuint64_t strides[2] = {cuuint64_t(o.ld) * 2, cuuint64_t(o.planes > 1 ? o.plane_stride : o.ld * o.rows) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(box_rows), 1}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// C [rows, cols] = A B^T over `depth`; the epilogue's fields of p are set by the caller.
template <int EPI, bool A_MN, bool B_MN, typename T, int PLANES, int TN>
qk_status launch_planes(const Call& c, ProductArgs p, const Operand& a, const Operand& b, int64_t rows,
                         int64_t cols, int64_t depth, int splits, int split_steps) {
  const auto kernel = product_kernel<EPI, A_MN, B_MN, T, TN, PLANES>;
  static std::atomic<uint64_t> prepared{0};  // one bit a device
  const uint64_t bit = uint64_t(1) << (c.dev.index & 63);
  if (!(prepared.load(std::memory_order_acquire) & bit)) {
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, product_smem(TN, PLANES)) != cudaSuccess ||
        cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) {
      cudaGetLastError();
      return QK_ERR_LAUNCH;
    }
    // The warps' register shares are taken from what the launch holds; a build
    // that holds less would wait for the rest forever.
    if (fa.numRegs * kProductThreads < kSplitRegisters) return QK_ERR_LAUNCH;
    prepared.fetch_or(bit, std::memory_order_acq_rel);
  }
  p.rows = int32_t(rows);
  p.cols = int32_t(cols);
  p.chunk = PLANES == 3 ? 2 : 16;
  p.depth = int32_t(depth);
  p.steps = int32_t(ceil_div(depth, kStepK));
  p.m_tiles = int32_t(ceil_div(rows, kTileM));
  p.n_tiles = int32_t(ceil_div(cols, TN));
  // The last column tile as a product of the columns it has: halves of whole
  // 8-row groups of B (64-column boxes where B is MN-major).
  const int64_t rest = cols - int64_t(p.n_tiles - 1) * TN, unit = B_MN ? 128 : 32;
  p.last_n = TN < 256 ? TN : int32_t(std::min<int64_t>(TN, round_up(rest, unit)));
  p.n_full = p.last_n == TN ? p.n_tiles : p.n_tiles - 1;
  p.split_steps = splits == 1 ? p.steps : split_steps;
  p.splits = int32_t(ceil_div(p.steps, p.split_steps));
  p.timeout_ns = kWaitTimeoutNs;
  p.status = c.dev.status;
  CUtensorMap ma, mb;
  if (!make_map(&ma, a, A_MN ? kStepK : 128) || !make_map(&mb, b, B_MN ? kStepK : TN / 2)) return QK_ERR_LAUNCH;
  const int64_t tiles = int64_t(p.m_tiles) * p.n_tiles * p.splits;
  if (tiles > INT32_MAX) return QK_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(unsigned(2 * std::min<int64_t>(tiles, std::min(kPairs, c.dev.sms / 2))), 1, 1);
  cfg.blockDim = dim3(kProductThreads, 1, 1);
  cfg.dynamicSmemBytes = product_smem(TN, PLANES);
  cfg.stream = static_cast<cudaStream_t>(c.stream);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, ma, mb, p) != cudaSuccess) {
    cudaGetLastError();
    return QK_ERR_LAUNCH;
  }
  return QK_OK;
}

// bf16 operands, or float32 ones in three planes.
template <int EPI, bool A_MN, bool B_MN, typename T, int TN = kTileN>
qk_status launch_product(const Call& c, const ProductArgs& p, const Operand& a, const Operand& b, int64_t rows,
                         int64_t cols, int64_t depth, int splits, int split_steps) {
  if constexpr (TN == kTileN && (sizeof(T) == 4 || EPI == kEpiLse)) {
    if (a.planes == 3)
      return launch_planes<EPI, A_MN, B_MN, T, 3, TN>(c, p, a, b, rows, cols, depth, splits, split_steps);
  }
  if constexpr (sizeof(T) == 2 || EPI == kEpiAccum)
    return launch_planes<EPI, A_MN, B_MN, T, 1, TN>(c, p, a, b, rows, cols, depth, splits, split_steps);
  return QK_ERR_UNSUPPORTED;  // not reached: float outputs have float operands
}

unsigned blocks(const Call& c, int64_t n) { return unsigned(std::min<int64_t>(ceil_div(n, 256), 32 * c.dev.sms)); }

// Rows that TMA reads where they are: bf16, 16-byte aligned.
bool in_place(const void* h, const void* w, int64_t K, int dtype) {
  return dtype == QK_BF16 && K % 8 == 0 && aligned16(h) && aligned16(w);
}

// `rows` rows of h or w as an operand, by way of the workspace at `at` if `copied`.
template <typename T>
qk_status operand(const Call& c, const Layout& l, bool copied, const T* src, int64_t rows, char* at, Operand* o) {
  *o = {src, c.K, rows, c.K, 1, 0};
  if (!copied) return QK_OK;
  *o = {at, c.K, rows, l.kp, l.planes, rows * l.kp};
  const dim3 grid(unsigned(std::min<int64_t>(ceil_div(rows, 8), 16 * c.dev.sms)));
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(at);
  if constexpr (sizeof(T) == 4) {
    if (c.K % 4 == 0 && aligned16(src))
      return launch_pdl(planes_kernel<T, true>, grid, 256, 0, c.stream, src, rows, int32_t(c.K), out, int32_t(l.kp),
                        rows * l.kp);
  }
  return launch_pdl(planes_kernel<T, false>, grid, 256, 0, c.stream, src, rows, int32_t(c.K), out, int32_t(l.kp),
                    rows * l.kp);
}

// Launches of the fp32 kernels for few tokens.
template <int MT, int KV, bool GRAD>
qk_status launch_few_logits(const Call& c, const Layout& l, const FewArgs& a) {
  const auto kernel = few_logits_kernel<float, MT, KV, GRAD>;
  static std::atomic<uint64_t> prepared{0};  // one bit a device
  const uint64_t bit = uint64_t(1) << (c.dev.index & 63);
  if (!(prepared.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kFewSmem)) != cudaSuccess) {
      cudaGetLastError();
      return QK_ERR_LAUNCH;
    }
    prepared.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_pdl(kernel, dim3(unsigned(l.few_grid)), kFewLogitThreads, size_t(MT) * size_t(a.chunk) * 4, c.stream, a);
}
template <bool GRAD>
qk_status few_logits(const Call& c, const Layout& l, const FewArgs& a) {
  const bool vec = c.K % 4 == 0 && aligned16(c.w);
  switch (l.few) {
    case 4: return vec ? launch_few_logits<4, 4, GRAD>(c, l, a) : launch_few_logits<4, 1, GRAD>(c, l, a);
    case 8: return vec ? launch_few_logits<8, 4, GRAD>(c, l, a) : launch_few_logits<8, 1, GRAD>(c, l, a);
    case 16: return vec ? launch_few_logits<16, 4, GRAD>(c, l, a) : launch_few_logits<16, 1, GRAD>(c, l, a);
    default: return vec ? launch_few_logits<32, 4, GRAD>(c, l, a) : launch_few_logits<32, 1, GRAD>(c, l, a);
  }
}
qk_status few_forward(const Call& c, const Layout& l, float* loss, float* lse, float* mean) {
  FewArgs f = {};
  f.h = c.h, f.w = c.w, f.V = c.V, f.M = int32_t(c.M), f.K = int32_t(c.K), f.chunk = l.few_chunk;
  f.targets = c.targets;
  f.part = reinterpret_cast<float2*>(c.ws + l.part);
  f.at_target = reinterpret_cast<float*>(c.ws + l.at_target);
  const qk_status st = few_logits<false>(c, l, f);
  if (st != QK_OK) return st;
  const LossArgs a = {f.part, c.M, l.few_grid, f.at_target, c.targets, c.M, c.V, c.has_ignore, c.z, c.ignore, loss,
                      lse, mean};
  return launch_pdl(join_few_kernel, dim3(1), 1024, 0, c.stream, a);
}
qk_status few_backward(const Call& c, const Layout& l, void* dh, void* dw) {
  FewArgs a = {};
  a.h = c.h, a.w = c.w, a.V = c.V, a.M = int32_t(c.M), a.K = int32_t(c.K), a.chunk = l.few_chunk;
  a.row = reinterpret_cast<const XentRow*>(c.ws + l.row);
  a.scale = reinterpret_cast<const float*>(c.ws + l.scale);
  a.g = reinterpret_cast<float*>(c.ws + l.g);
  a.sum = dh != nullptr ? reinterpret_cast<float*>(c.ws + l.sum) : nullptr;
  a.dw = dw;
  a.ld = c.K;
  a.columns = l.columns;
  a.per_split = l.per_split;
  qk_status st = few_logits<true>(c, l, a);
  if (st != QK_OK || (dh == nullptr && dw == nullptr)) return st;
  // The vectors' alignment is known only here; without it a thread takes one
  // column after the other of the same number of threads' worth, in more CTAs.
  const bool vec = l.few_kv > 1 && aligned16(c.w) && aligned16(dw);
  const int kv = vec ? l.few_kv : 1;
  const dim3 grid(unsigned(ceil_div(ceil_div(c.K, kv), l.columns)), unsigned(l.splits_y));
  const auto go = [&](auto kernel) { return launch_pdl(kernel, grid, kFewThreads, 0, c.stream, a); };
  switch (l.few) {
    case 4: st = vec ? go(few_grad_kernel<float, 4, 4>) : go(few_grad_kernel<float, 4, 1>); break;
    case 8: st = vec ? go(few_grad_kernel<float, 8, 4>) : go(few_grad_kernel<float, 8, 1>); break;
    case 16: st = vec ? go(few_grad_kernel<float, 16, 2>) : go(few_grad_kernel<float, 16, 1>); break;
    default: st = go(few_grad_kernel<float, 32, 1>);
  }
  if (st != QK_OK || dh == nullptr) return st;
  // Hundreds of splits of few sums: a warp for each 32 of them and every 32nd split.
  return launch_pdl(dw_reduce_kernel<0>, dim3(unsigned(ceil_div(c.M * c.K, 32))), kDwReduceThreads, 0, c.stream, a.sum,
                    static_cast<float*>(dh), l.splits, c.M * c.K);
}

template <typename T>
qk_status forward(const Call& c, int dtype, float* loss, float* lse, float* mean) {
  const bool copied = !in_place(c.h, c.w, c.K, dtype);
  const Layout& l = layout(false, c.M, c.V, c.K, dtype, copied);
  if (l.few != 0) return few_forward(c, l, loss, lse, mean);
  Operand h, w;
  qk_status st = operand(c, l, copied, static_cast<const T*>(c.h), c.M, c.ws + l.h, &h);
  ProductArgs p = {};
  p.targets = c.targets;
  p.part = reinterpret_cast<float2*>(c.ws + l.part);
  p.part_ld = c.M;
  p.at_target = reinterpret_cast<float*>(c.ws + l.at_target);
  int64_t pairs = 2 * ceil_div(c.V, kTileN);  // of a row, for the join
  const bool by_columns = c.M <= kFewTokens && l.planes == 1;
  if (by_columns) pairs = 0;
  for (p.v0 = 0; p.v0 < c.V && st == QK_OK; p.v0 += l.piece) {
    const int64_t width = std::min(l.piece, c.V - p.v0);
    st = operand(c, l, copied, static_cast<const T*>(c.w) + p.v0 * c.K, width, c.ws + l.w, &w);
    if (st != QK_OK) break;
    if (!by_columns) {
      st = launch_product<kEpiLse, false, false, __nv_bfloat16>(c, p, h, w, c.M, width, c.K, 1, 0);
      continue;
    }
    p.part0 = pairs / 2;
    st = c.M <= 16   ? launch_product<kEpiLseCols, false, false, __nv_bfloat16, 16>(c, p, w, h, width, c.M, c.K, 1, 0)
         : c.M <= 32 ? launch_product<kEpiLseCols, false, false, __nv_bfloat16, 32>(c, p, w, h, width, c.M, c.K, 1, 0)
                     : launch_product<kEpiLseCols, false, false, __nv_bfloat16, 64>(c, p, w, h, width, c.M, c.K, 1, 0);
    pairs += 2 * std::min<int64_t>(ceil_div(width, kTileM), std::min(kPairs, c.dev.sms / 2));
  }
  if (st != QK_OK) return st;
  const LossArgs a = {p.part, p.part_ld, pairs, p.at_target, c.targets, c.M, c.V, c.has_ignore, c.z, c.ignore, loss, lse,
                      mean};
  if (by_columns) return launch_pdl(join_few_kernel, dim3(1), 1024, 0, c.stream, a);
  st = launch_pdl(join_kernel, dim3(unsigned(ceil_div(c.M, 32))), 1024, 0, c.stream, a);
  if (st != QK_OK || mean == nullptr) return st;
  return launch_pdl(xent_mean_kernel<0>, dim3(1), 1024, 0, c.stream, loss, c.targets, c.M, c.has_ignore, c.ignore,
                    mean);
}

template <typename T>
qk_status backward(const Call& c, int dtype, const float* lse, const float* dloss, void* dh, void* dw) {
  const bool copied = !in_place(c.h, c.w, c.K, dtype);
  const Layout& l = layout(true, c.M, c.V, c.K, dtype, copied);
  XentRow* row = reinterpret_cast<XentRow*>(c.ws + l.row);
  float* scale = reinterpret_cast<float*>(c.ws + l.scale);
  float* sum = reinterpret_cast<float*>(c.ws + l.sum);
  const bool direct = l.piece >= c.V && l.splits == 1;  // dh is complete in one product
  Operand h, w, ht = {};
  qk_status st = launch_pdl(rows_kernel, dim3(1), 1024, 0, c.stream, c.targets, lse, dloss, c.M, c.V, c.has_ignore,
                            c.ignore, c.z, row, scale);
  if (l.few != 0) return st == QK_OK ? few_backward(c, l, dh, dw) : st;
  if (st == QK_OK) st = operand(c, l, copied, static_cast<const T*>(c.h), c.M, c.ws + l.h, &h);
  if (st == QK_OK && dw != nullptr && l.turned) {
    const int64_t ld = round_up(c.M, 8);
    ht = {c.ws + l.ht, c.M, c.K, ld, l.planes, c.K * ld};
    st = launch_pdl(transpose_kernel, dim3(unsigned(ceil_div(c.M, 64)), unsigned(ceil_div(c.K, 64)), unsigned(l.planes)),
                    256, 0, c.stream, static_cast<const uint16_t*>(h.base), c.M, c.K, h.ld, h.plane_stride,
                    reinterpret_cast<uint16_t*>(c.ws + l.ht), ld, c.K * ld);
  }
  for (int64_t v0 = 0; v0 < c.V && st == QK_OK; v0 += l.piece) {
    const int64_t width = std::min(l.piece, c.V - v0);
    st = operand(c, l, copied, static_cast<const T*>(c.w) + v0 * c.K, width, c.ws + l.w, &w);
    ProductArgs p = {};
    p.v0 = v0;
    p.row = row;
    p.out = c.ws + l.g;
    p.ld = l.ld_g;
    p.plane_stride = c.M * l.ld_g;
    if (st == QK_OK) st = launch_product<kEpiGrad, false, false, T>(c, p, h, w, c.M, width, c.K, 1, 0);
    const Operand g = {c.ws + l.g, width, c.M, l.ld_g, l.planes, c.M * l.ld_g};
    p = ProductArgs{};
    p.scale = scale;
    if (st == QK_OK && dh != nullptr) {
      p.vec = aligned16(dh) && c.K * int64_t(sizeof(T)) % 16 == 0;
      const bool last = l.splits == 1 && v0 + width == c.V;
      if (direct || last) {  // complete: rounded into dh
        p.out = dh;
        p.ld = c.K;
        p.sum = sum;
        p.sum_ld = l.kp;
        st = direct ? launch_product<kEpiStore, false, true, T>(c, p, g, w, c.M, c.K, width, 1, 0)
                    : launch_product<kEpiFinish, false, true, T>(c, p, g, w, c.M, c.K, width, 1, 0);
      } else {
        p.out = sum;
        p.ld = l.kp;
        p.first = v0 == 0;
        st = launch_product<kEpiAccum, false, true, float>(c, p, g, w, c.M, c.K, width, l.splits, l.split_steps);
      }
    }
    if (st == QK_OK && dw != nullptr) {
      p.out = static_cast<T*>(dw) + v0 * c.K;
      p.ld = c.K;
      p.vec = aligned16(dw) && c.K * int64_t(sizeof(T)) % 16 == 0;
      st = l.turned ? launch_product<kEpiStore, true, false, T>(c, p, g, ht, width, c.K, c.M, 1, 0)
                    : launch_product<kEpiStore, true, true, T>(c, p, g, h, width, c.K, c.M, 1, 0);
    }
  }
  if (st != QK_OK || dh == nullptr || l.splits == 1) return st;
  return launch_pdl(finish_kernel<T>, dim3(blocks(c, c.M * l.kp / 4)), 256, 0, c.stream, sum, int32_t(l.kp),
                    c.M * l.kp, l.splits, static_cast<T*>(dh), c.M, int32_t(c.K));
}

// Bytes that these sizes may need, whichever way the pointers are aligned.
qk_status workspace_size(bool bwd, int64_t M, int64_t V, int64_t K, int dtype, size_t* bytes) {
  if (bytes == nullptr) return QK_ERR_INVALID_ARG;
  *bytes = 0;
  const qk_status st = check_linear(dtype, M, V, K);
  if (st != QK_OK || M == 0) return st;
  *bytes = size_t(layout(bwd, M, V, K, dtype, true).total);
  if (dtype == QK_BF16) *bytes = std::max(*bytes, size_t(layout(bwd, M, V, K, dtype, false).total));
  return QK_OK;
}

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

qk_status qk_linear_xent_fwd_workspace_size(int64_t M, int64_t V, int64_t K, qk_dtype dtype, size_t* bytes) {
  return workspace_size(false, M, V, K, dtype, bytes);
}

qk_status qk_linear_xent_bwd_workspace_size(int64_t M, int64_t V, int64_t K, qk_dtype dtype, size_t* bytes) {
  return workspace_size(true, M, V, K, dtype, bytes);
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
  const Call c = {h, w, targets, M, V, K, has_ignore, ignore, z, static_cast<char*>(workspace), stream, d};
  if (M > 0)
    return dtype == QK_F32 ? forward<float>(c, dtype, loss, lse, mean_loss)
                           : forward<__nv_bfloat16>(c, dtype, loss, lse, mean_loss);
  if (mean_loss == nullptr) return QK_OK;
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
  const Call c = {h, w, targets, M, V, K, has_ignore, ignore, z, static_cast<char*>(workspace), stream, d};
  return dtype == QK_F32 ? backward<float>(c, dtype, lse, dloss, dh, dw)
                         : backward<__nv_bfloat16>(c, dtype, lse, dloss, dh, dw);
}

}  // extern "C"
