// qk_scaled_kernels.cuh -- 8-bit matrix products with a scale for each block of
// 128 (sm_103a, tcgen05).
//
//   y[i,j] = sum_c a_scale[i,c] b_scale[j',c] sum_{k in block c} a[i,k] b[j,k]
//
// The tensor cores form a block's sum of 128 k in TMEM (four products of 32 k,
// exact products of e4m3, fp32 sums); the epilogue warps take it out, multiply it
// with its two scales and add it to the running sum in registers, to nearest.
#pragma once

#include "qk_internal.h"
#include "qk_tensor.cuh"

namespace qk {

constexpr int kScaledThreads = 384;   // 4 warps that feed the tensor cores, 8 for the sums
constexpr int kScaledStepK = 128;     // k of a step: one block of the scales, 128 bytes
constexpr int kQuad = 4;              // steps whose scales travel together
constexpr int kScaleSlots = 4;        // quads of scales in shared memory
constexpr int kMaxExperts = 1024;

struct ScaledArgs {
  const float* a_scale;     // [M, groups]
  const float* b_scale;     // [experts][b rows >> b_shift][groups]
  const int32_t* offsets;   // [experts + 1], null: one group of M rows
  void* y;                  // [M, N]
  int64_t b_scale_stride;   // elements of one expert's scales
  int32_t M, N, groups;     // groups: blocks of 128 k, and steps
  int32_t experts;
  int32_t b_shift;          // 7: a scale a 128 rows of b, 0: a scale a row
  int32_t scale_vec;        // rows of scales are whole aligned float4
  int32_t lane_tiles;       // tiles along the axis that stands on TMEM's lanes
  int32_t split_steps;      // steps of one CTA of a cluster
  uint64_t timeout_ns;
  int* status;
};

// Where an expert's rows and tiles begin.  Offsets that fall or leave [0, M] are
// read as their running maximum within it, so no table leads out of bounds.
struct ExpertTable {
  int32_t row0[kMaxExperts + 1];
  int32_t tile0[kMaxExperts + 1];
};
// By one warp; `tile_rows` rows of a make a tile.
__device__ __forceinline__ void fill_table(ExpertTable& t, const ScaledArgs& p, int tile_rows, int lane) {
  if (p.offsets == nullptr) {
    if (lane == 0) {
      t.row0[0] = 0, t.row0[1] = p.M;
      t.tile0[0] = 0, t.tile0[1] = (p.M - 1) / tile_rows + 1;
    }
    return;
  }
  int32_t top = 0, tiles = 0;  // the running maximum and count before these 32
  for (int e0 = 0; e0 <= p.experts; e0 += 32) {
    const int e = e0 + lane;
    int32_t v = e <= p.experts ? min(max(p.offsets[e], 0), p.M) : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    v = max(v, top);
    // tiles of the expert in front of this offset
    int32_t before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = top;
    int32_t n = e == 0 ? 0 : (v - before + tile_rows - 1) / tile_rows;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int32_t u = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += u;
    }
    n += tiles;
    if (e <= p.experts) t.row0[e] = v, t.tile0[e] = n;
    top = __shfl_sync(0xffffffffu, v, 31);
    tiles = __shfl_sync(0xffffffffu, n, 31);
  }
}

// The scales of four steps for one row: zero behind the last.
__device__ __forceinline__ float4 load_quad(const float* row, int32_t s, int32_t end, bool vec) {
  if (vec) return *reinterpret_cast<const float4*>(row + s);  // groups is a multiple of 4
  return make_float4(row[s], s + 1 < end ? row[s + 1] : 0.f, s + 2 < end ? row[s + 2] : 0.f,
                     s + 3 < end ? row[s + 3] : 0.f);
}

// Shared memory of the tile kernel by its columns.
__host__ __device__ constexpr int tile_stage_bytes(int tn) { return (128 + tn) * kScaledStepK; }
__host__ __device__ constexpr int tile_stages(int tn) {
  return 196608 / tile_stage_bytes(tn) < 10 ? 196608 / tile_stage_bytes(tn) : 10;
}
__host__ __device__ constexpr int tile_slot_bytes(int tn) { return (128 + tn) * kQuad * 4; }
__host__ __device__ constexpr int tile_smem(int tn) {  // and room to start on 1024 bytes
  return tile_stages(tn) * tile_stage_bytes(tn) + kScaleSlots * tile_slot_bytes(tn) + 1024;
}

// ---------------------------------------------------------------------------
// Tiles of 128 rows of b x TN rows of a, one CTA each: b on TMEM's lanes, so that
// a few tokens are a few columns.  A cluster splits the k axis of one tile; its
// partial sums are joined through the CTAs' shared memory in rank order.
// ---------------------------------------------------------------------------
template <int TN, typename T>
__global__ void __launch_bounds__(kScaledThreads, 1)
    scaled_tile_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const ScaledArgs p) {
  constexpr int kStages = tile_stages(TN), kStageBytes = tile_stage_bytes(TN), kSlotBytes = tile_slot_bytes(TN);
  constexpr int kBufs = 4;
  constexpr uint32_t kColumns = kBufs * TN;
  constexpr int kCols = TN / 2 < 16 ? 16 : TN / 2, kReaders = 4 * (TN / kCols);
  extern __shared__ unsigned char dynamic_smem[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 2 * kBufs + 2 * kScaleSlots];
  __shared__ uint32_t tmem_at;
  __shared__ ExpertTable table;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * kStages, done0 = full0 + 16 * kStages,
                 free0 = done0 + 8 * kBufs, sfull0 = free0 + 8 * kBufs, sempty0 = sfull0 + 8 * kScaleSlots;
  const uint32_t ring = (smem_addr(dynamic_smem) + 1023u) & ~1023u;
  const uint32_t slots = ring + uint32_t(kStages * kStageBytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(done0 + 8 * i, 1);
      mbar_init(free0 + 8 * i, kReaders);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(sfull0 + 8 * i, 2);
      mbar_init(sempty0 + 8 * i, kReaders);
    }
    fence_mbar_init();
    prefetch_tensor_map(&map_a);
    prefetch_tensor_map(&map_b);
  }
  __syncwarp();
  if (warp == 2) {
    tmem_alloc(smem_addr(&tmem_at), kColumns);
    tmem_relinquish();
  }
  grid_dependency_wait();
  allow_dependent_launch();
  if (warp == 3) fill_table(table, p, TN, lane);
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_at;

  const int32_t tiles = table.tile0[p.experts] * p.lane_tiles;  // the host bounds it
  const int32_t first = int32_t(cluster_id_x()), step = int32_t(num_clusters_x());
  const int32_t s0 = int32_t(cluster_ctarank()) * p.split_steps, s1 = min(p.groups, s0 + p.split_steps);
  struct At {
    int32_t e, n0, row0, rows;  // expert, first row of b, first row of a, rows of a
  };
  // Tile t, for t that rise: the expert is found by walking on from the last.
  auto tile = [&](int32_t t, int32_t& e) {
    while (t >= table.tile0[e + 1] * p.lane_tiles) ++e;
    const int32_t in = t - table.tile0[e] * p.lane_tiles, m_tiles = table.tile0[e + 1] - table.tile0[e];
    At r;
    r.e = e;
    const int32_t n = in / m_tiles, m = in - n * m_tiles;
    r.n0 = n * 128;
    r.row0 = table.row0[e] + m * TN;
    r.rows = min(TN, table.row0[e + 1] - r.row0);
    return r;
  };

  bool failed = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_wait<false>(bar, parity, p.timeout_ns)) return true;
    report_status(p.status, 5);
    failed = true;
    return false;
  };

  float v[kCols];
  int32_t e = 0;
  if (warp == 0 && lane == 0) {
    // ---- producer ----
    int64_t q = 0;
    int st = 0;
    uint32_t turn = 0;
    for (int32_t t = first; t < tiles && !failed; t += step) {
      const At at = tile(t, e);
      for (int32_t s = s0; s < s1; ++s, ++q) {
        if (!wait(empty0 + 8 * st, turn ^ 1u)) break;
        const uint32_t bar = full0 + 8 * st, dst = ring + uint32_t(st) * kStageBytes;
        mbar_arrive_expect_tx(bar, kStageBytes);
        tma_load_3d_cta(dst, &map_b, s * kScaledStepK, at.n0, at.e, bar);
        tma_load_3d_cta(dst + 128 * kScaledStepK, &map_a, s * kScaledStepK, at.row0, 0, bar);
        if (++st == kStages) st = 0, turn ^= 1u;
      }
    }
    if (failed)  // leave once the loads in flight have landed
      for (int64_t i = max(int64_t(0), q - kStages); i < q; ++i)
        mbar_wait<false>(full0 + 8 * uint32_t(i % kStages), uint32_t(i / kStages) & 1u, p.timeout_ns);
  } else if (warp == 1 && lane == 0) {
    // ---- products ----
    constexpr uint32_t idesc = instruction_desc_e4m3(128, TN);
    int st = 0;
    uint32_t turn = 0, it = 0;
    for (int32_t t = first; t < tiles && !failed; t += step) {
      for (int32_t s = s0; s < s1; ++s, ++it) {
        const uint32_t buf = it % kBufs;
        if (!wait(free0 + 8 * buf, ((it / kBufs) & 1u) ^ 1u)) break;
        if (!wait(full0 + 8 * st, turn)) break;
        tcgen05_fence_after();
        const uint32_t sb = ring + uint32_t(st) * kStageBytes;
        const uint64_t db = operand_desc(sb, 0), da = operand_desc(sb + 128 * kScaledStepK, 0);
#pragma unroll
        for (int k = 0; k < kScaledStepK / 32; ++k)
          mma_e4m3(tmem + buf * TN, db + uint64_t(2 * k), da + uint64_t(2 * k), idesc, k > 0);
        mma_commit(empty0 + 8 * st);
        mma_commit(done0 + 8 * buf);
        if (++st == kStages) st = 0, turn ^= 1u;
      }
    }
  } else if (warp == 2 || warp == 3) {
    // ---- scales, four steps at a time: [128 rows of b][4], [4][TN rows of a] ----
    const int id = (warp - 2) * 32 + lane;
    uint32_t it = 0;
    for (int32_t t = first; t < tiles && !failed; t += step) {
      const At at = tile(t, e);
      const float* bs = p.b_scale + at.e * p.b_scale_stride;
      for (int32_t s = s0; s < s1; s += kQuad, ++it) {
        const uint32_t slot = it % kScaleSlots;
        const bool ok = wait(sempty0 + 8 * slot, ((it / kScaleSlots) & 1u) ^ 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        const uint32_t dst = slots + slot * kSlotBytes;
        const bool vec = p.scale_vec && (s & 3) == 0;
        float4 f[2], g[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = id + 64 * i;
          f[i] = g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (at.n0 + r < p.N) f[i] = load_quad(bs + int64_t((at.n0 + r) >> p.b_shift) * p.groups, s, s1, vec);
          if (r < at.rows) g[i] = load_quad(p.a_scale + int64_t(at.row0 + r) * p.groups, s, s1, vec);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = id + 64 * i;
          st_shared_v4(dst + r * 16, f[i]);
          if (r < TN) {
            const uint32_t c = dst + 128 * 16 + r * 4;
            st_shared(c, g[i].x);
            st_shared(c + TN * 4, g[i].y);
            st_shared(c + TN * 8, g[i].z);
            st_shared(c + TN * 12, g[i].w);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sfull0 + 8 * slot);
      }
    }
  } else if (warp >= 4 && warp < 4 + kReaders) {
    // ---- sums: half the tokens of a row of b a thread ----
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    uint32_t it = 0, sit = 0;
    for (int32_t t = first; t < tiles && !failed; t += step) {
      const At at = tile(t, e);
#pragma unroll
      for (int j = 0; j < kCols; ++j) v[j] = 0.f;
      for (int32_t q0 = s0; q0 < s1 && !failed; q0 += kQuad, ++sit) {
        const uint32_t slot = sit % kScaleSlots, src_s = slots + slot * kSlotBytes;
        bool ok = wait(sfull0 + 8 * slot, (sit / kScaleSlots) & 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        const float4 bq = ld_shared_v4(src_s + (quarter * 32 + lane) * 16);
        const float bs[4] = {bq.x, bq.y, bq.z, bq.w};
#pragma unroll
        for (int qi = 0; qi < kQuad; ++qi) {
          if (q0 + qi >= s1) break;
          const uint32_t buf = it % kBufs;
          ok = wait(done0 + 8 * buf, (it / kBufs) & 1u);
          if (!__all_sync(0xffffffffu, ok)) {
            failed = true;
            break;
          }
          ++it;
          tcgen05_fence_after();
          float x[kCols];
          const uint32_t src = tmem + (uint32_t(quarter * 32) << 16) + buf * TN + uint32_t(half * kCols);
#pragma unroll
          for (int c = 0; c < kCols; c += 16) tmem_load_16(src + uint32_t(c), x + c);
#pragma unroll
          for (int c = 0; c < kCols; c += 16) tmem_load_wait(x + c);
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(free0 + 8 * buf);
          const uint32_t sa = src_s + 128 * 16 + qi * (TN * 4) + half * (kCols * 4);
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            const float4 as = ld_shared_v4(sa + c * 4);
            // (sum a_scale) b_scale + running sum
            v[c] = fmaf(x[c] * as.x, bs[qi], v[c]);
            v[c + 1] = fmaf(x[c + 1] * as.y, bs[qi], v[c + 1]);
            v[c + 2] = fmaf(x[c + 2] * as.z, bs[qi], v[c + 2]);
            v[c + 3] = fmaf(x[c + 3] * as.w, bs[qi], v[c + 3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty0 + 8 * slot);
      }
      if (failed) break;
      if (cluster_nctarank() == 1) {
        const int32_t n = at.n0 + quarter * 32 + lane;
        if (n < p.N) {
          T* y = static_cast<T*>(p.y) + int64_t(at.row0) * p.N + n;
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            if (half * kCols + j < at.rows) Vec16<T>::store1(y + int64_t(half * kCols + j) * p.N, v[j]);
        }
      } else {
        // Every product of this CTA is done, so the ring is free: [TN][128] partial sums.
#pragma unroll
        for (int j = 0; j < kCols; ++j)
          st_shared(ring + uint32_t((half * kCols + j) * 128 + quarter * 32 + lane) * 4, v[j]);
      }
    }
  }
  __syncwarp();
  if (__syncthreads_or(failed)) {
    // Something was waited for in vain: give products and loads still under way
    // time to land before this CTA's memory goes to another (a bounded pause).
    failed = true;
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  const int32_t ranks = int32_t(cluster_nctarank());
  if (ranks > 1) {  // one tile a cluster
    cluster_sync_all();
    if (first < tiles && !failed && warp >= 4) {
      e = 0;
      const At at = tile(first, e);
      const int col = int(threadIdx.x) - 128;
      const int32_t n = at.n0 + (col & 127);
      // rank r takes tokens r, r + ranks, ...; two tokens at a time on 256 threads
      for (int j = (int(cluster_ctarank()) + (col >> 7) * ranks); j < at.rows; j += 2 * ranks) {
        float sum = 0.f;
        for (int32_t r = 0; r < ranks; ++r)
          sum += ld_shared_cluster(map_to_rank(ring + uint32_t(j * 128 + (col & 127)) * 4, uint32_t(r)));
        if (n < p.N) Vec16<T>::store1(static_cast<T*>(p.y) + int64_t(at.row0 + j) * p.N + n, sum);
      }
    }
    __syncwarp();
    cluster_sync_all();  // the others have read this CTA's sums
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp == 2) tmem_dealloc(tmem, kColumns);
}

// Rows of `cols` bytes that start anywhere, to rows of `ld` bytes (a multiple of
// 16) that start on 16: what TMA can read.  Bytes behind a row are not written.
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint8_t* in, int64_t rows, int32_t cols, uint8_t* out,
                                                       int32_t ld) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  for (int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); row < rows; row += int64_t(gridDim.x) * 8) {
    const uint8_t* src = in + row * cols;
    uint8_t* dst = out + row * ld;
    for (int32_t c = lane * 4; c < cols; c += 128) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < cols) w |= uint32_t(src[c + i]) << (8 * i);
      *reinterpret_cast<uint32_t*>(dst + c) = w;
    }
  }
}

}  // namespace qk
