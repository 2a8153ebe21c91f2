// qk_experts.cu -- tokens sorted by expert, and back with weights.
//
//   sort     offsets[e] = number of choices of experts below e; slot[t, j] = place
//            of choice (t, j) among the choices sorted by expert, in their order
//   gather   rows[slot[t, j]] = x[t]
//   combine  y[t] = sum_j weight[t, j] rows[slot[t, j]];
//            drows[slot[t, j]] = weight[t, j] dy[t],  dweight[t, j] = dy[t] . rows[slot[t, j]]
//
// All bound by memory (the sort by latency): a token's row is read once and its
// k rows are written, or the other way round.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "../../include/qk.h"
#include "qk_device.cuh"
#include "qk_host.h"

namespace qk {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int64_t kMaxChoices = INT32_MAX - 65536;
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
struct SortArgs {
  const void* ids;
  int32_t wide;       // ids are int64
  int32_t experts;
  int32_t blocks;
  int64_t n, chunk;   // choices, and those of a CTA
  int32_t* offsets;   // [experts + 1]
  int32_t* slot;      // [n]
  int32_t* counts;    // [blocks][experts], null where one CTA has all
};

__device__ __forceinline__ int32_t expert_at(const SortArgs& a, int64_t i) {
  const int64_t v = a.wide ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
  return v >= 0 && v < a.experts ? int32_t(v) : -1;
}

// Choices of each expert among a CTA's.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a) {
  __shared__ int32_t hist[kMaxExperts];
  grid_dependency_wait();
  allow_dependent_launch();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int64_t i0 = blockIdx.x * a.chunk, i1 = min(a.n, i0 + a.chunk);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
    const int32_t e = expert_at(a, i);
    if (e >= 0) atomicAdd(&hist[e], 1);  // whole numbers: any order gives the same
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) a.counts[int64_t(blockIdx.x) * a.experts + e] = hist[e];
}

// Places.  Each warp has a run of the CTA's choices: its counts by expert, summed
// over the warps before it, are where its first choice of an expert goes.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortArgs a) {
  extern __shared__ int32_t next[];  // [warps][experts]
  __shared__ int32_t sums[kSortWarps];
  grid_dependency_wait();
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = a.experts;
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) next[i] = 0;
  __syncthreads();
  const int64_t c0 = blockIdx.x * a.chunk, c1 = min(a.n, c0 + a.chunk);
  const int64_t run = ((a.chunk + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t i0 = min(c1, c0 + warp * run), i1 = min(c1, i0 + run);
  int32_t* mine = next + warp * E;
  for (int64_t i = i0 + lane; i < i1; i += 32) {
    const int32_t e = expert_at(a, i);
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  // Two experts a thread: all choices of each, those of the CTAs before this one, and
  // the sum over the experts below.
  int32_t total[2], before[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int e = int(threadIdx.x) * 2 + k;
    total[k] = before[k] = 0;
    if (e >= E) continue;
    if (a.counts != nullptr) {
      for (int b = 0; b < a.blocks; ++b) {
        const int32_t c = a.counts[int64_t(b) * E + e];
        total[k] += c;
        if (b < int(blockIdx.x)) before[k] += c;
      }
    } else {
      for (int w = 0; w < kSortWarps; ++w) total[k] += next[w * E + e];
    }
  }
  int32_t sum = total[0] + total[1];
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int32_t u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  if (lane == 31) sums[warp] = sum;
  __syncthreads();
  int32_t base = sum - total[0] - total[1];
  for (int w = 0; w < warp; ++w) base += sums[w];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int e = int(threadIdx.x) * 2 + k;
    if (e < E) {
      if (blockIdx.x == 0) {
        a.offsets[e] = base;
        if (e == E - 1) a.offsets[E] = base + total[k];
      }
      int32_t at = base + before[k];
      for (int w = 0; w < kSortWarps; ++w) {
        const int32_t c = next[w * E + e];
        next[w * E + e] = at;
        at += c;
      }
    }
    base += total[k];
  }
  __syncthreads();
  for (int64_t i = i0; i < i1; i += 32) {  // in order, 32 at a time
    const int32_t e = i + lane < i1 ? expert_at(a, i + lane) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int32_t at = e >= 0 ? mine[e] + rank : -1;
    __syncwarp();
    if (e >= 0 && rank == 0) mine[e] += __popc(same);
    __syncwarp();
    if (i + lane < i1) a.slot[i + lane] = at;
  }
}

// ---------------------------------------------------------------------------
// Gather: a warp copies a piece of a token's row to the places of its choices
// ---------------------------------------------------------------------------
struct GatherArgs {
  const uint8_t* x;
  const float* scale;
  const int32_t* slot;
  uint8_t* rows;
  float* row_scale;
  int64_t T, P, row_bytes, pieces;
  int32_t k, groups;
};

template <typename W, int WORDS>
__global__ void __launch_bounds__(256) gather_kernel(const GatherArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t words = a.row_bytes / int64_t(sizeof(W)), units = a.T * a.pieces;
  for (int64_t u = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units; u += int64_t(gridDim.x) * 8) {
    const int64_t t = u / a.pieces, piece = u - t * a.pieces;
    const W* src = reinterpret_cast<const W*>(a.x + t * a.row_bytes);
    const int64_t w0 = piece * (32 * WORDS) + lane;
    W v[WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
      if (w0 + 32 * i < words) v[i] = src[w0 + 32 * i];
    for (int j0 = 0; j0 < a.k; j0 += 32) {  // the places of 32 choices, a lane each
      const int count = min(32, a.k - j0);
      const int32_t place = lane < count ? a.slot[t * a.k + j0 + lane] : -1;
      for (int j = 0; j < count; ++j) {
        const int32_t at = __shfl_sync(0xffffffffu, place, j);
        if (at < 0 || at >= a.P) continue;
        W* dst = reinterpret_cast<W*>(a.rows + int64_t(at) * a.row_bytes);
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
          if (w0 + 32 * i < words) dst[w0 + 32 * i] = v[i];
      }
      if (piece != 0) continue;
      for (int g0 = 0; g0 < a.groups; g0 += 32) {
        const int g = g0 + lane;
        const float s = g < a.groups ? a.scale[t * a.groups + g] : 0.f;
        for (int j = 0; j < count; ++j) {
          const int32_t at = __shfl_sync(0xffffffffu, place, j);
          if (at >= 0 && at < a.P && g < a.groups) a.row_scale[int64_t(at) * a.groups + g] = s;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Combine
// ---------------------------------------------------------------------------
struct CombineArgs {
  const void* dy;        // [T, N] backward
  const void* rows;      // [P, N]
  const int32_t* slot;   // [T, k]
  const float* weights;  // [T, k], null: 1 (forward)
  void* out;             // [T, N] y, or [P, N] drows
  float* dweights;       // [T, k] backward, may be null
  int64_t T, P, N, pieces;
  int32_t k;
};

// A lane's 16 bytes of a row of N values, from a warp's piece of 512 bytes that begins at
// value `piece`: one vector where rows consist of those (WORD 16; the caller leaves
// lanes behind the row out), else words of 4 or 2 bytes.  ACROSS: a warp's lanes have
// neighbouring words, so that stores touch whole sectors (16384 x 4 of 4095 bf16,
// backward: 367 us, with a lane's words side by side 799).  Side by side suits
// loads of 2 bytes, whose first brings what the others need (forward: 220 and 313 us).
template <typename T, int WORD>
using Word = std::conditional_t<WORD == 16, uint4, std::conditional_t<WORD == 4, uint32_t, uint16_t>>;
template <typename T, int WORD, bool ACROSS>
__device__ __forceinline__ int word_at(int lane, int i) {  // the i-th word's first value in the piece
  constexpr int kWords = 16 / WORD, kValues = WORD / int(sizeof(T));
  return (ACROSS ? lane + 32 * i : kWords * lane + i) * kValues;
}
template <typename T, int WORD, bool ACROSS>
__device__ __forceinline__ uint4 load_raw(const T* row, int64_t piece, int lane, int64_t N) {
  using W = Word<T, WORD>;
  const T* p = row + piece;
  if constexpr (WORD == 16) {
    return *reinterpret_cast<const W*>(p + word_at<T, WORD, ACROSS>(lane, 0));
  } else {
    const int left = int(min(int64_t(512 / sizeof(T)), N - piece));  // values of the piece
    W v[16 / WORD];
#pragma unroll
    for (int i = 0; i < 16 / WORD; ++i) {
      const int at = word_at<T, WORD, ACROSS>(lane, i);
      v[i] = at < left ? *reinterpret_cast<const W*>(p + at) : W(0);
    }
    if constexpr (WORD == 4) return make_uint4(v[0], v[1], v[2], v[3]);
    else
      return make_uint4(v[0] | uint32_t(v[1]) << 16, v[2] | uint32_t(v[3]) << 16, v[4] | uint32_t(v[5]) << 16,
                        v[6] | uint32_t(v[7]) << 16);
  }
}
template <typename T, int WORD, bool ACROSS>
__device__ __forceinline__ void store_raw(T* row, int64_t piece, int lane, int64_t N, const float* f) {
  using W = Word<T, WORD>;
  const uint4 v = Vec16<T>::pack(f);
  T* p = row + piece;
  if constexpr (WORD == 16) {
    *reinterpret_cast<W*>(p + word_at<T, WORD, ACROSS>(lane, 0)) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const int left = int(min(int64_t(512 / sizeof(T)), N - piece));
#pragma unroll
    for (int i = 0; i < 16 / WORD; ++i) {
      const int at = word_at<T, WORD, ACROSS>(lane, i);
      if (at >= left) continue;
      if constexpr (WORD == 4) *reinterpret_cast<W*>(p + at) = w[i];
      else *reinterpret_cast<W*>(p + at) = W(w[i / 2] >> (16 * (i & 1)));
    }
  }
}

// Choices whose rows are loaded together.  16384 tokens of 4096 bf16, forward: four
// choices 113 us with 4, 126 with 2 (and 127 one after the other).
constexpr int kAtOnce = 4;

// A warp forms a piece of a token's row; the sum runs over the choices in order.
template <typename T, int WORD>
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs a) {
  constexpr int E = Vec16<T>::kElems;
  constexpr bool ACROSS = WORD != 2;
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const int64_t units = a.T * a.pieces;
  for (int64_t u = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units; u += int64_t(gridDim.x) * 8) {
    const int64_t t = u / a.pieces, piece = (u - t * a.pieces) * (32 * E);
    if (WORD == 16 && piece + lane * E >= a.N) continue;
    float sum[E] = {};
    for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
      int32_t at[kAtOnce];
      float w[kAtOnce];
      uint4 f[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        at[j] = j0 + j < a.k ? a.slot[t * a.k + j0 + j] : -1;
        if (at[j] >= a.P) at[j] = -1;
        w[j] = a.weights != nullptr && at[j] >= 0 ? a.weights[t * a.k + j0 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (at[j] >= 0) f[j] = load_raw<T, WORD, ACROSS>(static_cast<const T*>(a.rows) + int64_t(at[j]) * a.N, piece, lane, a.N);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (at[j] < 0) continue;
        float v[E];
        Vec16<T>::unpack(f[j], v);
#pragma unroll
        for (int i = 0; i < E; ++i) sum[i] = fmaf(w[j], v[i], sum[i]);
      }
    }
    store_raw<T, WORD, ACROSS>(static_cast<T*>(a.out) + t * a.N, piece, lane, a.N, sum);
  }
}

// THREADS threads take a token, AT choices at a time: dy and their rows are read
// together, drows leave at once, and each choice's products are summed over the
// threads at the end.  The registers are held down for the sake of CTAs an SM
// (16384 tokens of 4096 bf16, two choices: 142 us with three, 115 with five, 111
// with six and AT = 2; four choices: 201, 183, 189).
template <typename T, int WORD, int THREADS, int AT>
__global__ void __launch_bounds__(256, AT == 2 ? 6 : 5) combine_bwd_kernel(const CombineArgs a) {
  constexpr int E = Vec16<T>::kElems, kWarps = THREADS / 32, kTokens = 256 / THREADS;
  __shared__ float red[2][AT][kWarps];
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x % THREADS, warp = tid >> 5, lane = threadIdx.x & 31;
  int turn = 0;
  for (int64_t t = int64_t(blockIdx.x) * kTokens + threadIdx.x / THREADS; t < a.T; t += int64_t(gridDim.x) * kTokens) {
    const T* dy = static_cast<const T*>(a.dy) + t * a.N;
    for (int j0 = 0; j0 < a.k; j0 += AT) {
      int32_t at[AT];
      float w[AT], dot[AT] = {};
#pragma unroll
      for (int j = 0; j < AT; ++j) {
        at[j] = j0 + j < a.k ? a.slot[t * a.k + j0 + j] : -1;
        if (at[j] >= a.P) at[j] = -1;
        w[j] = at[j] >= 0 ? a.weights[t * a.k + j0 + j] : 0.f;
      }
      for (int64_t piece = warp * (32 * E); piece < a.N; piece += THREADS * E) {
        if (WORD == 16 && piece + lane * E >= a.N) break;
        const uint4 graw = load_raw<T, WORD, true>(dy, piece, lane, a.N);
        uint4 f[AT];
#pragma unroll
        for (int j = 0; j < AT; ++j)
          if (at[j] >= 0) f[j] = load_raw<T, WORD, true>(static_cast<const T*>(a.rows) + int64_t(at[j]) * a.N, piece, lane, a.N);
        float g[E];
        Vec16<T>::unpack(graw, g);
#pragma unroll
        for (int j = 0; j < AT; ++j) {
          if (at[j] < 0) continue;
          float v[E];
          Vec16<T>::unpack(f[j], v);
#pragma unroll
          for (int i = 0; i < E; ++i) {
            dot[j] = fmaf(g[i], v[i], dot[j]);
            v[i] = g[i] * w[j];
          }
          store_raw<T, WORD, true>(static_cast<T*>(a.out) + int64_t(at[j]) * a.N, piece, lane, a.N, v);
        }
      }
      if (a.dweights == nullptr) continue;
#pragma unroll
      for (int j = 0; j < AT; ++j) {
        if (j0 + j >= a.k) break;
        dot[j] = group_sum<32>(dot[j]);
        if (kWarps > 1 && lane == 0) red[turn][j][warp] = dot[j];
      }
      if constexpr (kWarps > 1) {
        __syncthreads();  // one is enough: the next sums go to the other half
        if (tid < AT && j0 + tid < a.k) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < kWarps; ++i) s += red[turn][tid][i];
          a.dweights[t * a.k + j0 + tid] = s;
        }
        turn ^= 1;
      } else if (lane == 0) {
#pragma unroll
        for (int j = 0; j < AT; ++j)
          if (j0 + j < a.k) a.dweights[t * a.k + j0 + j] = dot[j];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }

qk_status check_choices(int64_t T, int64_t k) {
  if (T < 0 || k <= 0) return QK_ERR_INVALID_ARG;
  if (T > kMaxChoices / k) return QK_ERR_UNSUPPORTED;
  return QK_OK;
}
// CTAs of a sort of n choices.  Up to 2048 one, in one launch (4096: 6.2 us, 5.0 in two
// launches of 4).  Beyond, each CTA adds up the counts of all: 32 CTAs where 1024 choices
// each are enough (16384: 5.5 us, with 2048 or 4096 each 6.1 and 7.8), 128 at most (65536:
// 7.2 us with 32 CTAs, 7.6 with 64; 524288: 13.3 with 128, 14.6 with 152).
int64_t sort_blocks(int64_t n) {
  if (n <= 2048) return 1;
  return n <= 32768 ? ceil_div(n, 1024) : std::min<int64_t>(128, ceil_div(n, 2048));
}

unsigned warps_grid(const CurrentDevice& d, int64_t units) {
  return unsigned(std::max<int64_t>(1, std::min<int64_t>(ceil_div(units, 8), int64_t(d.sms) * 32)));
}

struct Buffer {
  const void* p;
  int64_t n;
};
template <int NO, int NI>
bool any_overlap(const Buffer (&out)[NO], const Buffer (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (const Buffer& b : in)
      if (overlap(out[i].p, out[i].n, b.p, b.n)) return true;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
}

template <typename T, int WORD>
qk_status launch_combine(const CurrentDevice& d, bool bwd, const CombineArgs& a, void* stream) {
  if (!bwd) return launch_pdl(combine_kernel<T, WORD>, dim3(warps_grid(d, a.T * a.pieces)), 256, 0, stream, a);
  // A warp a token for rows of at most two vectors a lane, and of at most four where there
  // are 16 tokens for each SM; else a CTA.  us, bf16 with four choices, a warp and a CTA:
  // 9728 tokens of 512 14.0 and 31.4, of 1024 31.9 and 42.8, of 1536 46.6 and 50.6, of 2048
  // 61.1 and 59.1; 2432 of 1024 6.8 and 8.7, of 1023 20.4 and 21.1, of 1536 9.1 and 9.9; 608 of
  // 1024 4.8 and 3.5, of 512 3.5 and 3.1.
  const int64_t warp_values = 32 * Vec16<T>::kElems;
  const bool narrow = a.N <= 2 * warp_values || (a.N <= 4 * warp_values && a.T >= 16 * int64_t(d.sms));
  const auto kernel = a.k <= 2 ? (narrow ? combine_bwd_kernel<T, WORD, 32, 2> : combine_bwd_kernel<T, WORD, 256, 2>)
                               : (narrow ? combine_bwd_kernel<T, WORD, 32, 4> : combine_bwd_kernel<T, WORD, 256, 4>);
  const int64_t blocks = narrow ? ceil_div(a.T, 8) : a.T;
  return launch_pdl(kernel, dim3(unsigned(std::min<int64_t>(blocks, int64_t(d.sms) * 32))), 256, 0, stream, a);
}
// By the widest word that all rows consist of.
template <typename T>
qk_status launch_combine(const CurrentDevice& d, bool bwd, CombineArgs a, void* stream) {
  a.pieces = ceil_div(a.N, 32 * Vec16<T>::kElems);
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.rows) |
                        reinterpret_cast<uintptr_t>(a.out) | uintptr_t(a.N) * sizeof(T);
  if (all % 16 == 0) return launch_combine<T, 16>(d, bwd, a, stream);
  if constexpr (sizeof(T) == 2)
    if (all % 4 != 0) return launch_combine<T, 2>(d, bwd, a, stream);
  return launch_combine<T, 4>(d, bwd, a, stream);
}

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

qk_status qk_expert_sort_workspace_size(int64_t T, int64_t k, int64_t experts, size_t* bytes) {
  if (bytes == nullptr) return QK_ERR_INVALID_ARG;
  *bytes = 0;
  const qk_status st = check_choices(T, k);
  if (st != QK_OK) return st;
  if (experts <= 0) return QK_ERR_INVALID_ARG;
  if (experts > kMaxExperts) return QK_ERR_UNSUPPORTED;
  const int64_t blocks = sort_blocks(T * k);
  if (blocks > 1) *bytes = size_t(blocks * experts * 4);
  return QK_OK;
}

qk_status qk_expert_sort(const void* experts, int64_t id_bytes, int32_t* offsets, int32_t* slot, void* workspace,
                         size_t workspace_bytes, int64_t T, int64_t k, int64_t num_experts, void* stream) {
  size_t need = 0;
  qk_status st = qk_expert_sort_workspace_size(T, k, num_experts, &need);
  if (st != QK_OK) return st;
  if (id_bytes != 4 && id_bytes != 8) return QK_ERR_INVALID_ARG;
  const int64_t n = T * k;
  if (offsets == nullptr || (n > 0 && (experts == nullptr || slot == nullptr))) return QK_ERR_INVALID_ARG;
  if (!aligned_to(experts, size_t(id_bytes)) || !aligned_to(offsets, 4) || !aligned_to(slot, 4)) return QK_ERR_MISALIGNED;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return QK_ERR_INVALID_ARG;
    if (!aligned_to(workspace, 16)) return QK_ERR_MISALIGNED;
  }
  const Buffer out[] = {{offsets, (num_experts + 1) * 4}, {slot, n * 4}, {workspace, int64_t(need)}},
               in[] = {{experts, n * id_bytes}};
  if (any_overlap(out, in)) return QK_ERR_INVALID_ARG;
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  SortArgs a = {};
  a.ids = experts;
  a.wide = id_bytes == 8;
  a.experts = int32_t(num_experts);
  a.n = n;
  a.blocks = int32_t(std::max<int64_t>(1, sort_blocks(n)));
  a.chunk = ceil_div(std::max<int64_t>(n, 1), a.blocks);
  a.offsets = offsets;
  a.slot = slot;
  a.counts = a.blocks > 1 ? static_cast<int32_t*>(workspace) : nullptr;
  if (a.blocks > 1) {
    st = launch_pdl(sort_count_kernel, dim3(unsigned(a.blocks)), kSortThreads, 0, stream, a);
    if (st != QK_OK) return st;
  }
  const size_t smem = size_t(kSortWarps) * num_experts * 4;
  if (smem > (48 << 10) - 1024) {
    static std::atomic<uint64_t> prepared{0};  // one bit a device
    const uint64_t bit = uint64_t(1) << (d.index & 63);
    if (!(prepared.load(std::memory_order_acquire) & bit)) {
      if (cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSortWarps * kMaxExperts * 4) != cudaSuccess) {
        cudaGetLastError();
        return QK_ERR_LAUNCH;
      }
      prepared.fetch_or(bit, std::memory_order_acq_rel);
    }
  }
  return launch_pdl(sort_place_kernel, dim3(unsigned(a.blocks)), kSortThreads, smem, stream, a);
}

qk_status qk_expert_gather_fwd(const void* x, const float* scale, const int32_t* slot, void* rows, float* row_scale,
                               int64_t T, int64_t k, int64_t P, int64_t row_bytes, int64_t groups, void* stream) {
  qk_status st = check_choices(T, k);
  if (st != QK_OK) return st;
  if (P < 0 || row_bytes <= 0 || groups < 0) return QK_ERR_INVALID_ARG;
  if (P > INT32_MAX || groups > INT32_MAX) return QK_ERR_UNSUPPORTED;
  if (std::max(T, P) > INT64_MAX / 16 / std::max(row_bytes, groups)) return QK_ERR_UNSUPPORTED;
  if ((scale == nullptr) != (groups == 0) || (row_scale == nullptr) != (groups == 0)) return QK_ERR_INVALID_ARG;
  if (T == 0 || P == 0) return QK_OK;
  if (x == nullptr || slot == nullptr || rows == nullptr) return QK_ERR_INVALID_ARG;
  if (!aligned_to(scale, 4) || !aligned_to(slot, 4) || !aligned_to(row_scale, 4)) return QK_ERR_MISALIGNED;
  const Buffer out[] = {{rows, P * row_bytes}, {row_scale, P * groups * 4}},
               in[] = {{x, T * row_bytes}, {scale, T * groups * 4}, {slot, T * k * 4}};
  if (any_overlap(out, in)) return QK_ERR_INVALID_ARG;
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  GatherArgs a = {static_cast<const uint8_t*>(x), scale, slot, static_cast<uint8_t*>(rows), row_scale,
                  T, P, row_bytes, 0, int32_t(k), int32_t(groups)};
  // The widest word that rows consist of.
  const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(rows) | uintptr_t(row_bytes);
  auto launch = [&](auto many, auto few, int64_t word) {
    // Eight words a lane where that fills the GPU (16384 x 4 of 4096 bf16: 103 us, with four
    // words 105); two for a few rows, whose time is latency (16 x 4 of 4096 bytes:
    // 2.6 us, with eight 4.0).
    const int64_t words = row_bytes / word;
    const bool wide = T * ceil_div(words, 256) >= int64_t(d.sms) * 8;
    a.pieces = ceil_div(words, wide ? 256 : 64);
    return launch_pdl(wide ? many : few, dim3(warps_grid(d, T * a.pieces)), 256, 0, stream, a);
  };
  if (all % 16 == 0) return launch(gather_kernel<uint4, 8>, gather_kernel<uint4, 2>, 16);
  if (all % 4 == 0) return launch(gather_kernel<uint32_t, 8>, gather_kernel<uint32_t, 2>, 4);
  if (all % 2 == 0) return launch(gather_kernel<uint16_t, 8>, gather_kernel<uint16_t, 2>, 2);
  return launch(gather_kernel<uint8_t, 8>, gather_kernel<uint8_t, 2>, 1);
}

qk_status qk_expert_combine_fwd(const void* rows, const int32_t* slot, const float* weights, void* y, int64_t T,
                                int64_t k, int64_t P, int64_t N, qk_dtype dtype, void* stream) {
  qk_status st = check_choices(T, k);
  if (st != QK_OK) return st;
  if (dtype != QK_F32 && dtype != QK_BF16) return QK_ERR_INVALID_ARG;
  if (P < 0 || N <= 0) return QK_ERR_INVALID_ARG;
  if (P > INT32_MAX || std::max(T, P) > INT64_MAX / 16 / N) return QK_ERR_UNSUPPORTED;
  if (T == 0) return QK_OK;
  if ((rows == nullptr && P > 0) || slot == nullptr || y == nullptr) return QK_ERR_INVALID_ARG;
  const size_t es = size_t(elem_size(dtype));
  if (!aligned_to(rows, es) || !aligned_to(y, es) || !aligned_to(slot, 4) || !aligned_to(weights, 4))
    return QK_ERR_MISALIGNED;
  const Buffer out[] = {{y, T * N * int64_t(es)}},
               in[] = {{rows, P * N * int64_t(es)}, {slot, T * k * 4}, {weights, T * k * 4}};
  if (any_overlap(out, in)) return QK_ERR_INVALID_ARG;
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  const CombineArgs a = {nullptr, rows, slot, weights, y, nullptr, T, P, N, 0, int32_t(k)};
  return dtype == QK_F32 ? launch_combine<float>(d, false, a, stream) : launch_combine<__nv_bfloat16>(d, false, a, stream);
}

qk_status qk_expert_combine_bwd(const void* dy, const void* rows, const int32_t* slot, const float* weights,
                                void* drows, float* dweights, int64_t T, int64_t k, int64_t P, int64_t N,
                                qk_dtype dtype, void* stream) {
  qk_status st = check_choices(T, k);
  if (st != QK_OK) return st;
  if (dtype != QK_F32 && dtype != QK_BF16) return QK_ERR_INVALID_ARG;
  if (P < 0 || N <= 0) return QK_ERR_INVALID_ARG;
  if (P > INT32_MAX || std::max(T, P) > INT64_MAX / 16 / N) return QK_ERR_UNSUPPORTED;
  if (T == 0) return QK_OK;
  if (dy == nullptr || slot == nullptr || weights == nullptr || (P > 0 && (rows == nullptr || drows == nullptr)))
    return QK_ERR_INVALID_ARG;
  const size_t es = size_t(elem_size(dtype));
  if (!aligned_to(dy, es) || !aligned_to(rows, es) || !aligned_to(drows, es) || !aligned_to(slot, 4) ||
      !aligned_to(weights, 4) || !aligned_to(dweights, 4))
    return QK_ERR_MISALIGNED;
  const int64_t pb = P * N * int64_t(es);
  const Buffer out[] = {{drows, pb}, {dweights, T * k * 4}},
               in[] = {{dy, T * N * int64_t(es)}, {drows == rows ? nullptr : rows, pb}, {slot, T * k * 4},
                       {weights, T * k * 4}};
  if (any_overlap(out, in) || overlap(dweights, T * k * 4, rows, pb)) return QK_ERR_INVALID_ARG;
  CurrentDevice d;
  st = current_device(&d);
  if (st != QK_OK) return st;
  const CombineArgs a = {dy, rows, slot, weights, drows, dweights, T, P, N, 0, int32_t(k)};
  return dtype == QK_F32 ? launch_combine<float>(d, true, a, stream) : launch_combine<__nv_bfloat16>(d, true, a, stream);
}

}  // extern "C"
