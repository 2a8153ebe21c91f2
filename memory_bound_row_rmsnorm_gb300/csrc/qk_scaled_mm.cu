// qk_scaled_mm.cu -- 8-bit matrix products with a scale for each block of 128,
// of all rows with one set of weights or of rows sorted by expert with each
// expert's own.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/qk.h"
#include "qk_host.h"
#include "qk_scaled_kernels.cuh"
#include "qk_tensor_map.h"

namespace qk {
namespace {

constexpr int64_t kMaxDim = INT32_MAX - 15;  // TMA coordinates, and rows padded to 16, are 32-bit

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
  return QK_OK;
}

// Rows that TMA cannot read where they are go through the workspace.
int64_t copy_bytes(int64_t M, int64_t N, int64_t K, int64_t experts) {
  return K % 16 == 0 ? 0 : (M + N * experts) * round_up(K, 16);
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

constexpr int64_t kMostTiles = int64_t(1) << 30;  // tile numbers are 32-bit

template <int TN, typename T>
qk_status launch_tiles(const Call& c) {
  const auto kernel = scaled_tile_kernel<TN, T>;
  static std::atomic<uint64_t> prepared{0};  // one bit a device
  const qk_status st = prepare(prepared, c.dev, kernel, tile_smem(TN));
  if (st != QK_OK) return st;
  ScaledArgs p = arguments(c);
  p.n_tiles = int32_t(ceil_div(c.N, 128));
  const int64_t tiles = most_tiles(c, TN) * p.n_tiles;
  if (tiles > kMostTiles) return QK_ERR_UNSUPPORTED;
  // Where the tiles leave SMs idle, a cluster shares a tile's k.
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= c.dev.sms && p.groups >= ranks * 2) ranks *= 2;
  p.split_steps = int32_t(ceil_div(p.groups, ranks));
  CUtensorMap ma, mb;
  if (!make_map(&ma, c.a, c.K, c.M, 1, c.ld, TN) || !make_map(&mb, c.b, c.K, c.N, c.experts, c.ld, 128))
    return QK_ERR_LAUNCH;
  return launch(c, kernel, ranks > 1 ? tiles * ranks : std::min<int64_t>(tiles, c.dev.sms), kScaledThreads, ranks,
                tile_smem(TN), ma, mb, p);
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
  p.y_vec = c.N * int64_t(sizeof(T)) % 16 == 0 && aligned16(c.y);
  const int64_t tiles = most_tiles(c, 256) * p.n_tiles;
  if (tiles > kMostTiles) return QK_ERR_UNSUPPORTED;
  CUtensorMap ma, mb, my = {};
  if (!make_map(&ma, c.a, c.K, c.M, 1, c.ld, 128) || !make_map(&mb, c.b, c.K, c.N, c.experts, c.ld, 128) ||
      (p.y_vec && !make_out_map(&my, c, int(sizeof(T)))))
    return QK_ERR_LAUNCH;
  return launch(c, kernel, 2 * std::min<int64_t>(tiles, c.dev.sms / 2), kPairThreads, 2, pair_smem(COLS), ma, mb, my, p);
}

// Rows of a and b as TMA reads them, by way of the workspace where K is not a multiple of 16.
qk_status pad_operands(Call& c, void* workspace) {
  if (c.ld == c.K) return QK_OK;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  PadArgs p = {};
  p.rows[0] = c.N * c.experts;
  p.rows[1] = c.M;
  p.in[0] = static_cast<const uint8_t*>(c.b);
  p.in[1] = static_cast<const uint8_t*>(c.a);
  p.out[0] = at;
  p.out[1] = at + p.rows[0] * c.ld;
  p.cols = int32_t(c.K);
  p.ld = int32_t(c.ld);
  c.b = p.out[0];
  c.a = p.out[1];
  const unsigned grid = unsigned(std::min<int64_t>(ceil_div(p.rows[0] + p.rows[1], 8), 16 * c.dev.sms));
  return launch_pdl(pad_rows_kernel, dim3(grid), 256, 0, c.stream, p);
}

template <typename T>
qk_status product(const Call& c) {
  const int64_t mean = ceil_div(c.M, c.experts);  // rows of a group, as far as the host knows
  if (mean <= 16) return launch_tiles<16, T>(c);
  if (mean <= 32) return launch_tiles<32, T>(c);
  if (mean <= 64) return launch_tiles<64, T>(c);
  if (mean <= 256) return launch_tiles<128, T>(c);
  return c.b_rows == 1 ? launch_pairs<true, T>(c) : launch_pairs<false, T>(c);
}

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

qk_status qk_scaled_mm_workspace_size(int64_t M, int64_t N, int64_t K, int64_t experts, size_t* bytes) {
  if (bytes == nullptr) return QK_ERR_INVALID_ARG;
  *bytes = 0;
  const qk_status st = check_sizes(M, N, K, experts);
  if (st == QK_OK && M > 0) *bytes = size_t(copy_bytes(M, N, K, experts));
  return st;
}

qk_status qk_scaled_mm_fwd(const void* a, const float* a_scale, const void* b, const float* b_scale,
                           const int32_t* offsets, void* y, void* workspace, size_t workspace_bytes, int64_t M,
                           int64_t N, int64_t K, int64_t experts, int64_t b_block_rows, qk_dtype out_dtype,
                           void* stream) {
  qk_status st = check_sizes(M, N, K, experts);
  if (st != QK_OK) return st;
  if (out_dtype != QK_F32 && out_dtype != QK_BF16) return QK_ERR_INVALID_ARG;
  if (b_block_rows != 1 && b_block_rows != 128) return QK_ERR_INVALID_ARG;
  if (offsets == nullptr && experts != 1) return QK_ERR_INVALID_ARG;
  if (M == 0) return QK_OK;
  if (a == nullptr || a_scale == nullptr || b == nullptr || b_scale == nullptr || y == nullptr)
    return QK_ERR_INVALID_ARG;
  const size_t es = size_t(elem_size(out_dtype));
  if (!aligned_to(y, es) || !aligned_to(a_scale, 4) || !aligned_to(b_scale, 4) || !aligned_to(offsets, 4))
    return QK_ERR_MISALIGNED;
  if (K % 16 == 0 && (!aligned16(a) || !aligned16(b))) return QK_ERR_MISALIGNED;
  const int64_t need = copy_bytes(M, N, K, experts), groups = ceil_div(K, kScaledStepK);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < size_t(need)) return QK_ERR_INVALID_ARG;
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
