// qk_product_kernel.cuh -- matrix products on tcgen05 with the epilogues of the
// linear cross-entropy (sm_103a).
//
//   C[i,j] = sum_k A(i,k) B(j,k),  bf16 operands, fp32 sums
//
// What bounds it: the tensor cores.  A pair of CTAs forms a 256 x 256 tile; a
// step of 64 k is 4 products of 16 k and 64 KB of operands through TMA, so each
// byte that reaches shared memory is used 128 times.  Warp 0 keeps TMA loads
// six steps ahead, warp 1 of the leading CTA issues the products, warps 4-7
// turn the finished sums (TMEM holds two tiles) into outputs while the next
// tile is being summed.  The grid is persistent: one CTA an SM.
//
// An operand is stored with k innermost (K-major) or with its rows innermost
// (MN-major): h, w and g serve as either, without a transposed copy.
//
// float32 operands come as three bf16 planes, x = x0 + x1 + x2 with 8 bits of
// the significand each (what is left is below 2^-26 of x); the products x_a y_b
// with a + b <= 2 are summed, the small ones first, as one long k axis.  What is
// left out is below 2^-25 of a term.
#pragma once

#include "qk_internal.h"
#include "qk_tensor.cuh"

namespace qk {

constexpr int kProductThreads = 256;
constexpr int kTileM = 256;       // rows of a pair's tile
constexpr int kTileN = 256;       // most columns of one
constexpr int kStepK = 64;        // k of one pipeline step: 128 bytes
constexpr int kStages = 6;
constexpr int kOperandBytes = 128 * kStepK * 2;  // one CTA's part of A (or of B at 256 columns)
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kProductSmem = kStages * kStageBytes + 1024;  // and room to start on 1024 bytes

enum Epilogue : int { kEpiLse = 0, kEpiGrad = 1, kEpiAccum = 2, kEpiStore = 3 };

struct XentRow {   // what the gradient needs of a row
  float lse, g, zf;  // g: dloss / scale (NaN for a bad target); zf = 1 + 2 z lse
  int32_t target;    // -1: none, -2: an ignored row
};

struct ProductArgs {
  int32_t rows, cols;        // of C
  int32_t steps;             // steps of 64 k in one plane pair
  int32_t planes;            // 1 (bf16) or 3 (float32)
  int32_t m_tiles, n_tiles;
  int32_t splits, split_steps;  // the k axis in pieces of split_steps steps
  int32_t bn;                // columns of a tile
  uint64_t timeout_ns;
  int* status;
  // epilogues; v0: vocabulary index of column 0
  int64_t v0;
  const int64_t* targets;    // lse
  float2* part;              // lse: [column tile][part_ld] running (maximum, sum)
  int64_t part_ld;
  float* at_target;          // lse: logit of the target
  const XentRow* row;        // grad
  void* out;                 // grad: bf16 [planes][rows][ld]; accum: fp32 [splits][rows][ld]; store: [rows][ld]
  int64_t ld, plane_stride;  // elements
  int32_t first;             // accum: overwrite
  int32_t vec;               // store: rows start on 16 bytes
  const float* scale;        // store: factor (device)
};

// Splits a float into three bf16 parts; what is not finite stays in the first.
__device__ __forceinline__ void split3(float x, __nv_bfloat16* b) {
  b[0] = __float2bfloat16_rn(x);
  const float r1 = x - __bfloat162float(b[0]);
  const bool fin = fabsf(x) < __int_as_float(0x7f800000) && fabsf(r1) < __int_as_float(0x7f800000);
  b[1] = __float2bfloat16_rn(fin ? r1 : 0.f);
  b[2] = __float2bfloat16_rn(fin ? r1 - __bfloat162float(b[1]) : 0.f);
}

// Tile number -> (split, row tile, column tile).  Eight row tiles are walked
// together: the pairs that run at one time then share their operands in L2
// (76 pairs: 8 row tiles x 9.5 column tiles, a quarter of the loads unique).
struct TileAt {
  int split, m, n;
};
__device__ __forceinline__ TileAt tile_at(const ProductArgs& p, int64_t t) {
  const int64_t per = int64_t(p.m_tiles) * p.n_tiles;
  TileAt r;
  r.split = int(t / per);
  const int64_t in = t % per;
  const int64_t group = in / (int64_t(8) * p.n_tiles);
  const int64_t rest = in % (int64_t(8) * p.n_tiles);
  const int wide = min(8, p.m_tiles - int(group) * 8);
  r.m = int(group) * 8 + int(rest % wide);
  r.n = int(rest / wide);
  return r;
}

template <int EPI, bool A_MN, bool B_MN, typename T>
__global__ void __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const ProductArgs p) {
  extern __shared__ unsigned char dynamic_smem[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t tmem_at;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * kStages, done0 = full0 + 16 * kStages,
                 free0 = done0 + 16;
  const uint32_t ring = (smem_addr(dynamic_smem) + 1023u) & ~1023u;  // the same in both CTAs
  const int64_t tiles = int64_t(p.m_tiles) * p.n_tiles * p.splits;
  const int64_t first_tile = cluster_id_x(), tile_step = num_clusters_x();
  const int pairs = p.planes == 3 ? 6 : 1;
  const int total_steps = pairs * p.steps;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);   // the leader's producer, and the bytes of both CTAs
      mbar_init(empty0 + 8 * s, 1);  // a commit of the leader's products
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(done0 + 8 * i, 1);  // a commit: the tile is summed
      mbar_init(free0 + 8 * i, 8);  // four epilogue warps of each CTA have read it
    }
    fence_mbar_init();
    prefetch_tensor_map(&map_a);
    prefetch_tensor_map(&map_b);
  }
  __syncwarp();
  if (warp == 2) {
    tmem_alloc_pair(smem_addr(&tmem_at), 512);
    tmem_relinquish_pair();
  }
  tcgen05_fence_before();
  cluster_sync_all();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_at;
  grid_dependency_wait();
  allow_dependent_launch();

  bool failed = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_wait<true>(bar, parity, p.timeout_ns)) return true;
    report_status(p.status, 5);
    failed = true;
    return false;
  };

  if (warp == 0 && lane == 0) {
    // ---- producer: this CTA's half of each step's operands ----
    const int half_n = p.bn / 2;
    const uint32_t bytes = 2u * uint32_t(kOperandBytes + half_n * kStepK * 2);
    int64_t q = 0;  // steps issued
    for (int64_t t = first_tile; t < tiles && !failed; t += tile_step) {
      const TileAt at = tile_at(p, t);
      const int a0 = at.m * kTileM + int(rank) * 128, b0 = at.n * p.bn + int(rank) * half_n;
      const int s0 = at.split * p.split_steps, s1 = min(total_steps, s0 + p.split_steps);
      for (int s = s0; s < s1; ++s, ++q) {
        const int st = int(q % kStages);
        if (!wait(empty0 + 8 * st, (uint32_t(q / kStages) & 1u) ^ 1u)) break;
        const int pair = s / p.steps, k = (s % p.steps) * kStepK;
        // (2,0) (1,1) (0,2) (1,0) (0,1) (0,0): the small products first
        const int pa = pairs == 1 ? 0 : pair < 3 ? 2 - pair : pair == 3 ? 1 : 0;
        const int pb = pairs == 1 ? 0 : pair < 3 ? pair : pair == 4 ? 1 : 0;
        const uint32_t bar = map_to_rank(full0 + 8 * st, 0);
        if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * st, bytes);
        const uint32_t da = ring + uint32_t(st) * kStageBytes, db = da + kOperandBytes;
        if constexpr (A_MN) {
          tma_load_3d(da, &map_a, a0, k, pa, bar);
          tma_load_3d(da + kOperandBytes / 2, &map_a, a0 + 64, k, pa, bar);
        } else {
          tma_load_3d(da, &map_a, k, a0, pa, bar);
        }
        if constexpr (B_MN) {
          for (int i = 0; i < half_n / 64; ++i)
            tma_load_3d(db + uint32_t(i) * (64 * kStepK * 2), &map_b, b0 + 64 * i, k, pb, bar);
        } else {
          tma_load_3d(db, &map_b, k, b0, pb, bar);
        }
      }
    }
    // A failed launch leaves once the loads in flight have landed: the leader's
    // barriers count those of both CTAs.
    if (failed && rank == 0)
      for (int64_t i = max(int64_t(0), q - kStages); i < q; ++i)
        mbar_wait<true>(full0 + 8 * uint32_t(i % kStages), uint32_t(i / kStages) & 1u, p.timeout_ns);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- products of both CTAs ----
    const uint32_t idesc = instruction_desc(A_MN, B_MN, uint32_t(p.bn));
    constexpr uint32_t kLbo = 64 * kStepK * 2;                       // MN-major: the next 64 rows
    constexpr uint32_t kAStep = (A_MN ? 16 * 128 : 32) >> 4, kBStep = (B_MN ? 16 * 128 : 32) >> 4;  // 16 k
    int64_t q = 0;
    int it = 0;
    for (int64_t t = first_tile; t < tiles && !failed; t += tile_step, ++it) {
      const TileAt at = tile_at(p, t);
      const int s0 = at.split * p.split_steps, s1 = min(total_steps, s0 + p.split_steps);
      const int acc = it & 1;
      if (!wait(free0 + 8 * acc, ((uint32_t(it) >> 1) & 1u) ^ 1u)) break;
      tcgen05_fence_after();
      const uint32_t d = tmem + uint32_t(acc) * kTileN;
      for (int s = s0; s < s1; ++s, ++q) {
        const int st = int(q % kStages);
        if (!wait(full0 + 8 * st, uint32_t(q / kStages) & 1u)) break;
        tcgen05_fence_after();
        const uint32_t sa = ring + uint32_t(st) * kStageBytes;
        const uint64_t da = operand_desc(sa, A_MN ? kLbo : 0), db = operand_desc(sa + kOperandBytes, B_MN ? kLbo : 0);
#pragma unroll
        for (int k = 0; k < kStepK / 16; ++k)
          mma_bf16_pair(d, da + uint64_t(k) * kAStep, db + uint64_t(k) * kBStep, idesc, s > s0 || k > 0);
        mma_commit_pair(empty0 + 8 * st);
      }
      if (!failed) mma_commit_pair(done0 + 8 * acc);
    }
  } else if (warp >= 4) {
    // ---- epilogue: one row a thread ----
    const int quarter = warp & 3;
    int it = 0;
    for (int64_t t = first_tile; t < tiles; t += tile_step, ++it) {
      const TileAt at = tile_at(p, t);
      const int acc = it & 1;
      if (!wait(done0 + 8 * acc, (uint32_t(it) >> 1) & 1u)) break;
      tcgen05_fence_after();
      const int64_t i = int64_t(at.m) * kTileM + rank * 128 + quarter * 32 + lane;
      const int64_t j0 = int64_t(at.n) * p.bn;
      const bool live = i < p.rows;
      const int width = int(min(int64_t(p.bn), p.cols - j0));  // columns of C in this tile
      const uint32_t src = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(acc) * kTileN;

      XentRow row = {};
      int target = -1;  // column of the target in this tile
      if (live && EPI == kEpiLse) {
        const int64_t c = p.targets[i] - p.v0 - j0;
        target = c >= 0 && c < width ? int(c) : -1;
      }
      if (live && EPI == kEpiGrad) {
        row = p.row[i];
        const int64_t c = row.target - p.v0 - j0;
        target = row.target >= 0 && c >= 0 && c < width ? int(c) : -1;
      }
      float m = kNegInf, sum = 0.f;
      const float factor = EPI == kEpiStore ? *p.scale : 1.f;

      for (int c0 = 0; c0 < width; c0 += 32) {
        float v[32];
        __syncwarp();  // the load is a warp's; rows past the last skipped the output
        tmem_load_32(src + uint32_t(c0), v);
        if constexpr (EPI == kEpiLse) {
          // a running maximum and sum of exponentials; columns past the last are -inf
          if (width - c0 < 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = j < width - c0 ? v[j] : kNegInf;
          }
          if (unsigned(target - c0) < 32u) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j == target - c0) p.at_target[i] = v[j];
          }
          float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int j = 4; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], v[j]);
          const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          // All -inf so far: shift by 0, so that a NaN among them still shows.
          const float base = mn == kNegInf ? 0.f : mn * kLog2e;
          float s[4] = {};
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j & 3] += exp2_approx(fmaf(v[j], kLog2e, -base));
          sum = (m == kNegInf ? sum : sum * exp2_approx(fmaf(m, kLog2e, -base))) + ((s[0] + s[1]) + (s[2] + s[3]));
          m = mn;
        } else if constexpr (EPI == kEpiGrad) {
          if (live) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float g = exp2_approx((v[j] - row.lse) * kLog2e) * row.zf;
              if (j == target - c0) g -= 1.f;
              v[j] = row.target == -2 ? 0.f : g * row.g;
            }
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + i * p.ld + j0 + c0;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              if (c0 + j >= width) break;  // ld is a multiple of 8: whole vectors stay inside the row
              if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint4*>(out + j) = Vec16<__nv_bfloat16>::pack(v + j);
              } else {
                __nv_bfloat16 b[8][3];
#pragma unroll
                for (int e = 0; e < 8; ++e) split3(v[j + e], b[e]);
#pragma unroll
                for (int pl = 0; pl < 3; ++pl) {
                  __align__(16) __nv_bfloat16 o[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e) o[e] = b[e][pl];
                  *reinterpret_cast<uint4*>(out + pl * p.plane_stride + j) = *reinterpret_cast<const uint4*>(o);
                }
              }
            }
          }
        } else if constexpr (EPI == kEpiAccum) {
          if (live) {
            float* out = static_cast<float*>(p.out) + (int64_t(at.split) * p.rows + i) * p.ld + j0 + c0;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              if (c0 + j >= width) break;  // ld is a multiple of 4
              float4* o = reinterpret_cast<float4*>(out + j);
              float4 x = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
              if (!p.first) {
                const float4 y = *o;
                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
              }
              *o = x;
            }
          }
        } else {
          if (live) {
            T* out = static_cast<T*>(p.out) + i * p.ld + j0 + c0;
            constexpr int E = Vec16<T>::kElems;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= factor;
            if (p.vec) {
#pragma unroll
              for (int j = 0; j < 32; j += E)
                if (c0 + j < width) *reinterpret_cast<uint4*>(out + j) = Vec16<T>::pack(v + j);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (c0 + j < width) Vec16<T>::store1(out + j, v[j]);
            }
          }
        }
      }
      tcgen05_fence_before();
      __syncwarp();  // all lanes have read their sums
      if (lane == 0) mbar_arrive_cluster(map_to_rank(free0 + 8 * acc, 0));
      if (EPI == kEpiLse && live)
        p.part[(p.v0 / p.bn + at.n) * p.part_ld + i] = make_float2(m, sum);
    }
  }
  __syncwarp();
  if (__syncthreads_or(failed)) {
    // Something was waited for in vain: give products and loads still under way
    // time to land before this CTA's memory goes to another (a bounded pause).
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  tcgen05_fence_before();
  cluster_sync_all();
  tcgen05_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem, 512);
}

}  // namespace qk
