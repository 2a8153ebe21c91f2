// qk_scaled_mm.cu -- 8-bit matrix products with a scale for each block of 128,
// of all rows with one set of weights or of rows sorted by expert with each
// expert's own.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/qk.h"
#include "qk_host.h"
#include "qk_scaled_kernels.cuh"
#include "qk_tensor_map.h"

namespace qk {
namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;  // TMA coordinates, a tile's behind the last row too, are 32-bit
constexpr int64_t kMostTiles = int64_t(1) << 30;         // and so are tile numbers

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }

struct Call {
  const void* a;
  const float* a_scale;
  const void* b;
  const float* b_scale;
  const int32_t* offsets;
  void* y;
  int64_t M, N, K, experts, b_rows;
  int64_t ld;  // bytes of a row of a and b as TMA reads them
  void* stream;
  CurrentDevice dev;
};

qk_status check_sizes(int64_t M, int64_t N, int64_t K, int64_t experts) {
  if (M < 0 || N <= 0 || K <= 0 || experts <= 0) return QK_ERR_INVALID_ARG;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim || experts > kMaxExperts) return QK_ERR_UNSUPPORTED;
  if (std::max(M, N * experts) > INT64_MAX / 1024 / std::max(N, K)) return QK_ERR_UNSUPPORTED;  // byte offsets fit int64
  if (ceil_div(N, 256) > kMostTiles / (ceil_div(M, 256) + experts)) return QK_ERR_UNSUPPORTED;
  return QK_OK;
}

qk_status check_call(const int32_t* offsets, int64_t M, int64_t N, int64_t K, int64_t experts, int64_t b_block_rows,
                     qk_dtype out_dtype) {
  const qk_status st = check_sizes(M, N, K, experts);
  if (st != QK_OK) return st;
  if (out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_ARG;
  if (b_block_rows != 1 && b_block_rows != 128) return QK_ERR_INVALID_ARG;
  return offsets == nullptr && experts != 1 ? QK_ERR_INVALID_ARG : QK_OK;
}

// Rows that TMA cannot read where they are go through the workspace: all where K is
// not a multiple of 16, else those of an operand that starts off 16 bytes.
bool copied(const void* operand, int64_t K) { return K % 16 != 0 || !aligned16(operand); }
int64_t copy_bytes(const void* a, const void* b, int64_t M, int64_t N, int64_t K, int64_t experts) {
  return ((copied(a, K) ? M : 0) + (copied(b, K) ? N * experts : 0)) * round_up(K, 16);
}

// Rows of bytes [planes][rows][ld] of which the first `inner` count, in boxes of
// 128 x box_rows in 128-byte swizzle; what lies outside reads as zero.
bool make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t rows, int64_t planes, int64_t ld,
              int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(rows), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(ld), cuuint64_t(ld * rows)};
  const cuuint32_t box[3] = {kScaledStepK, cuuint32_t(box_rows), 1}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y in boxes of 32 rows of 128 bytes, for stores.
bool make_out_map(CUtensorMap* map, const Call& c, int es) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {cuuint64_t(c.N), cuuint64_t(c.M)};
  const cuuint64_t strides[1] = {cuuint64_t(c.N) * cuuint64_t(es)};
  const cuuint32_t box[2] = {cuuint32_t(128 / es), 32}, steps[2] = {1, 1};
  return encode(map, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.y, dims,
                strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Once a device and kernel: its shared memory, and whether the launch holds the
// registers that its warps share out (a build that held less would wait for the
// rest forever).
template <typename K>
qk_status prepare(std::atomic<uint64_t>& prepared, const CurrentDevice& d, K kernel, int smem, int threads = 0,
                  int registers = 0) {
  const uint64_t bit = uint64_t(1) << (d.index & 63);
  if (prepared.load(std::memory_order_acquire) & bit) return QK_OK;
  cudaFuncAttributes fa;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) {
    cudaGetLastError();
    return QK_ERR_LAUNCH;
  }
  if (fa.numRegs * threads < registers) return QK_ERR_LAUNCH;
  prepared.fetch_or(bit, std::memory_order_acq_rel);
  return QK_OK;
}

// Most tiles of `rows` rows that M rows in this many groups can make.
int64_t most_tiles(const Call& c, int64_t rows) {
  if (c.offsets == nullptr) return ceil_div(c.M, rows);
  return std::min(c.M, c.M / rows + c.experts);
}

ScaledArgs arguments(const Call& c) {
  ScaledArgs p = {};
  p.a_scale = c.a_scale;
  p.b_scale = c.b_scale;
  p.offsets = c.offsets;
  p.y = c.y;
  p.M = int32_t(c.M);
  p.N = int32_t(c.N);
  p.groups = int32_t(ceil_div(c.K, kScaledStepK));
  p.experts = int32_t(c.experts);
  p.b_shift = c.b_rows == 1 ? 0 : 7;
  p.b_scale_stride = ceil_div(c.N, c.b_rows) * p.groups;
  p.scale_vec = p.groups % 4 == 0 && aligned16(c.a_scale) && aligned16(c.b_scale);
  p.timeout_ns = kWaitTimeoutNs;
  p.status = c.dev.status;
  return p;
}

template <typename K, typename... A>
qk_status launch(const Call& c, K kernel, int64_t grid, int threads, int cluster, int smem, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(unsigned(grid), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = static_cast<cudaStream_t>(c.stream);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return QK_ERR_LAUNCH;
  }
  return QK_OK;
}

// Clusters of 2, 4 and 8 CTAs of a tile kernel that a device holds at a time
// (clusters lie within a GPC, so 8 take fewer of the SMs).
struct Clusters {
  std::atomic<int> most[3] = {{0}, {0}, {0}};
};
template <typename K>
int most_clusters(Clusters& known, const CurrentDevice& d, K kernel, int log2_size, int smem) {
  std::atomic<int>& slot = known.most[log2_size - 1];
  int n = slot.load(std::memory_order_relaxed);  // devices of one kind: what one answers holds for all
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(unsigned(d.sms / 8 * 8), 1, 1);
    cfg.blockDim = dim3(kScaledThreads, 1, 1);
    cfg.dynamicSmemBytes = size_t(smem);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log2_size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    n = std::max(n, 1);
    slot.store(n, std::memory_order_relaxed);
  }
  return n;
}

// How the tile kernel of TN columns would do a call, and about how long it would take.
struct TilePlan {
  qk_status status;
  int64_t tiles;  // at most
  int ranks;      // CTAs that share a tile's k
  double us;
};

// Tiles of `rows` rows that M rows in groups of unknown sizes make, about: half of
// the groups that have rows have a tile more than their share, and each has one.
double likely_tiles(const Call& c, int64_t rows) {
  if (c.offsets == nullptr) return double(ceil_div(c.M, rows));
  const double active = double(std::min(c.M, c.experts));
  return std::max(active, double(c.M) / double(rows) + 0.5 * active);
}

// Microseconds: a launch, and a step and an end for each tile that an SM does one
// after the other.  Measured over 1 to 2048 rows x 200 to 8192 x 1024 to 8192, and
// 2 to 16384 rows of 32 experts x 4096 x 2048 and 2048 x 4096, in a graph.
constexpr double kTileLaunch = 5.2, kPairLaunch = 4.4, kPairStep = 0.40, kPairStepRows = 0.59;
constexpr double kTileEndF32 = 1.45;  // times the end in bf16
// A pair's tile's end, bf16 and float32: rows of y on 16 bytes, which leave by TMA, and off them.
constexpr double kPairEnd[2] = {1.7, 3.0}, kPairEndOff[2] = {3.2, 5.2};
template <int TN>
constexpr double tile_step() { return TN == 16 ? 0.24 : TN == 32 ? 0.25 : TN == 64 ? 0.28 : 0.41; }
template <int TN>
constexpr double tile_end() { return TN == 16 ? 0.8 : TN == 32 ? 1.0 : TN == 64 ? 1.1 : 3.2; }

template <int TN, typename T>
TilePlan plan_tiles(const Call& c) {
  const auto kernel = scaled_tile_kernel<TN, T>;
  static std::atomic<uint64_t> prepared{0};  // one bit a device
  static Clusters known;
  TilePlan plan = {};
  plan.status = prepare(prepared, c.dev, kernel, tile_smem(TN));
  if (plan.status != QK_OK) return plan;
  const int64_t n_tiles = ceil_div(c.N, 128), groups = ceil_div(c.K, kScaledStepK);
  plan.tiles = most_tiles(c, TN) * n_tiles;
  // Where the tiles leave SMs idle, a cluster shares a tile's k: the largest of
  // which all run at one time (1 x 2048 x 8192: 12.9 us with 16 clusters of 8, of
  // which not all do, 9.1 with clusters of 4).
  int log2_ranks = 0;
  while (log2_ranks < 3 && groups >= 2 << log2_ranks && plan.tiles * (2 << log2_ranks) <= c.dev.sms &&
         plan.tiles <= most_clusters(known, c.dev, kernel, log2_ranks + 1, tile_smem(TN)))
    ++log2_ranks;
  plan.ranks = 1 << log2_ranks;
  const double waves = std::ceil(likely_tiles(c, TN) * double(n_tiles) * plan.ranks / c.dev.sms);
  plan.us = kTileLaunch + waves * (double(ceil_div(groups, plan.ranks)) * tile_step<TN>() + tile_end<TN>() * (sizeof(T) == 4 ? kTileEndF32 : 1.0));
  return plan;
}

int64_t tiles_grid(const Call& c, const TilePlan& plan) {
  return plan.ranks > 1 ? plan.tiles * plan.ranks : std::min<int64_t>(plan.tiles, c.dev.sms);
}
int64_t pairs_grid(const Call& c) {
  return 2 * std::min<int64_t>(most_tiles(c, 256) * ceil_div(c.N, 256), c.dev.sms / 2);
}

template <int TN, typename T>
qk_status launch_tiles(const Call& c, const TilePlan& plan) {
  ScaledArgs p = arguments(c);
  p.n_tiles = int32_t(ceil_div(c.N, 128));
  p.split_steps = int32_t(ceil_div(p.groups, plan.ranks));
  CUtensorMap ma, mb;
  if (!make_map(&ma, c.a, c.K, c.M, 1, c.ld, TN) || !make_map(&mb, c.b, c.K, c.N, c.experts, c.ld, 128))
    return QK_ERR_LAUNCH;
  return launch(c, scaled_tile_kernel<TN, T>, tiles_grid(c, plan), kScaledThreads, plan.ranks, tile_smem(TN), ma, mb, p);
}

// Rows of y are whole 16-byte vectors, which leave by TMA.
template <typename T>
bool whole_rows(const Call& c) {
  return c.N * int64_t(sizeof(T)) % 16 == 0 && aligned16(c.y);
}

template <bool COLS, typename T>
qk_status launch_pairs(const Call& c) {
  const auto kernel = scaled_pair_kernel<COLS, T>;
  static std::atomic<uint64_t> prepared{0};  // one bit a device
  const qk_status st = prepare(prepared, c.dev, kernel, pair_smem(COLS), kPairThreads, kSplitRegistersPair);
  if (st != QK_OK) return st;
  ScaledArgs p = arguments(c);
  p.n_tiles = int32_t(ceil_div(c.N, 256));
  // The last column tile as a product of the columns it has: halves of whole 8-row groups of b.
  p.last_n = int32_t(std::min<int64_t>(256, round_up(c.N - int64_t(p.n_tiles - 1) * 256, 32)));
  p.n_full = p.last_n == 256 ? p.n_tiles : p.n_tiles - 1;
  p.y_vec = whole_rows<T>(c);
  CUtensorMap ma, mb, my = {};
  if (!make_map(&ma, c.a, c.K, c.M, 1, c.ld, 128) || !make_map(&mb, c.b, c.K, c.N, c.experts, c.ld, 128) ||
      (p.y_vec && !make_out_map(&my, c, int(sizeof(T)))))
    return QK_ERR_LAUNCH;
  return launch(c, kernel, pairs_grid(c), kPairThreads, 2, pair_smem(COLS), ma, mb, my, p);
}

// Rows of a and b as TMA reads them, by way of the workspace where it has to be.
qk_status pad_operands(Call& c, void* workspace) {
  const bool copy_a = copied(c.a, c.K), copy_b = copied(c.b, c.K);
  if (!copy_a && !copy_b) return QK_OK;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  PadArgs p = {};
  p.rows[0] = copy_b ? c.N * c.experts : 0;
  p.rows[1] = copy_a ? c.M : 0;
  p.in[0] = static_cast<const uint8_t*>(c.b);
  p.in[1] = static_cast<const uint8_t*>(c.a);
  p.out[0] = at;
  p.out[1] = at + p.rows[0] * c.ld;
  p.offsets = c.offsets;
  p.M = c.M;
  p.experts = int32_t(c.experts);
  p.expert_rows = int32_t(c.N);
  p.cols = int32_t(c.K);
  p.ld = int32_t(c.ld);
  if (copy_b) c.b = p.out[0];
  if (copy_a) c.a = p.out[1];
  const unsigned grid = unsigned(std::min<int64_t>(ceil_div(p.rows[0] + p.rows[1], 8), 16 * c.dev.sms));
  return launch_pdl(pad_rows_kernel, dim3(grid), 256, 0, c.stream, p);
}

// Which kernel does a call: a plan of tiles, or pairs (pick -1).
struct Choice {
  qk_status status;
  int pick;
  TilePlan plans[4];  // 16, 32, 64 and 128 rows of a
};
template <typename T>
Choice choose(const Call& c) {
  Choice r = {QK_OK, -1, {plan_tiles<16, T>(c), plan_tiles<32, T>(c), plan_tiles<64, T>(c), plan_tiles<128, T>(c)}};
  const double waves = std::ceil(likely_tiles(c, 256) * double(ceil_div(c.N, 256)) / (c.dev.sms / 2));
  const double step = c.b_rows == 1 ? kPairStepRows : kPairStep;
  const double end = (whole_rows<T>(c) ? kPairEnd : kPairEndOff)[sizeof(T) == 4];
  double best = kPairLaunch + waves * (double(ceil_div(c.K, kScaledStepK)) * step + end);
  for (int i = 0; i < 4; ++i) {
    if (r.plans[i].status != QK_OK) {
      r.status = r.plans[i].status;
      return r;
    }
    if (r.plans[i].us < best && r.plans[i].tiles <= kMostTiles) best = r.plans[i].us, r.pick = i;
  }
  return r;
}

template <typename T>
qk_status product(const Call& c) {
  const Choice r = choose<T>(c);
  if (r.status != QK_OK) return r.status;
  switch (r.pick) {
    case 0: return launch_tiles<16, T>(c, r.plans[0]);
    case 1: return launch_tiles<32, T>(c, r.plans[1]);
    case 2: return launch_tiles<64, T>(c, r.plans[2]);
    case 3: return launch_tiles<128, T>(c, r.plans[3]);
    default: return c.b_rows == 1 ? launch_pairs<true, T>(c) : launch_pairs<false, T>(c);
  }
}

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

qk_status qk_scaled_mm_workspace_size(int64_t M, int64_t N, int64_t K, int64_t experts, size_t* bytes) {
  if (bytes == nullptr) return QK_ERR_INVALID_ARG;
  *bytes = 0;
  const qk_status st = check_sizes(M, N, K, experts);
  if (st == QK_OK && M > 0) *bytes = size_t(copy_bytes(nullptr, nullptr, M, N, K, experts));
  return st;
}

qk_status qk_scaled_mm_get_plan(const int32_t* offsets, const void* y, int64_t M, int64_t N, int64_t K,
                                int64_t experts, int64_t b_block_rows, qk_dtype out_dtype, qk_scaled_mm_plan* plan) {
  if (plan == nullptr) return QK_ERR_INVALID_ARG;
  *plan = {};
  qk_status st = check_call(offsets, M, N, K, experts, b_block_rows, out_dtype);
  if (st != QK_OK || M == 0) return st;
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  const Call c = {nullptr, nullptr, nullptr, nullptr, offsets, const_cast<void*>(y), M, N, K, experts, b_block_rows,
                  round_up(K, 16), nullptr, d};
  const Choice r = out_dtype == QK_F32 ? choose<float>(c) : choose<__nv_bfloat16>(c);
  if (r.status != QK_OK) return r.status;
  const bool pairs = r.pick < 0;
  plan->rows = pairs ? 256 : 16 << r.pick;
  plan->columns = pairs ? 256 : 128;
  plan->ctas = pairs ? 2 : r.plans[r.pick].ranks;
  plan->grid = int32_t(pairs ? pairs_grid(c) : tiles_grid(c, r.plans[r.pick]));
  return QK_OK;
}

qk_status qk_scaled_mm_fwd(const void* a, const float* a_scale, const void* b, const float* b_scale,
                           const int32_t* offsets, void* y, void* workspace, size_t workspace_bytes, int64_t M,
                           int64_t N, int64_t K, int64_t experts, int64_t b_block_rows, qk_dtype out_dtype,
                           void* stream) {
  qk_status st = check_call(offsets, M, N, K, experts, b_block_rows, out_dtype);
  if (st != QK_OK || M == 0) return st;
  if (a == nullptr || a_scale == nullptr || b == nullptr || b_scale == nullptr || y == nullptr)
    return QK_ERR_INVALID_ARG;
  const size_t es = size_t(elem_size(out_dtype));
  if (!aligned_to(y, es) || !aligned_to(a_scale, 4) || !aligned_to(b_scale, 4) || !aligned_to(offsets, 4))
    return QK_ERR_MISALIGNED;
  const int64_t need = copy_bytes(a, b, M, N, K, experts), groups = ceil_div(K, kScaledStepK);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < size_t(need))
      return K % 16 == 0 ? QK_ERR_MISALIGNED : QK_ERR_INVALID_ARG;
    if (!aligned_to(workspace, 256)) return QK_ERR_MISALIGNED;
  }
  const struct {
    const void* p;
    int64_t n;
  } in[] = {{a, M * K},
            {a_scale, M * groups * 4},
            {b, experts * N * K},
            {b_scale, experts * ceil_div(N, b_block_rows) * groups * 4},
            {offsets, (experts + 1) * 4}};
  for (const auto& i : in)
    if (overlap(y, M * N * int64_t(es), i.p, i.n) || overlap(workspace, need, i.p, i.n)) return QK_ERR_INVALID_ARG;
  if (overlap(y, M * N * int64_t(es), workspace, need)) return QK_ERR_INVALID_ARG;
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  Call c = {a, a_scale, b, b_scale, offsets, y, M, N, K, experts, b_block_rows, round_up(K, 16), stream, d};
  st = pad_operands(c, workspace);
  if (st != QK_OK) return st;
  return out_dtype == QK_F32 ? product<float>(c) : product<__nv_bfloat16>(c);
}

}  // extern "C"
