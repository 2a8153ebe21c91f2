// qk_scaled_kernels.cuh -- 8-bit matrix products with a scale for each block of
// 128 (sm_103a, tcgen05).
//
//   y[i,j] = sum_c a_scale[i,c] b_scale[j',c] sum_{k in block c} a[i,k] b[j,k]
//
// The tensor cores form a block's sum of 128 k in TMEM (four products of 32 k,
// exact products of e4m3, fp32 sums); the epilogue warps take it out, multiply it
// with its two scales and add it to the running sum in registers, to nearest.
#pragma once

#include <type_traits>

#include "qk_internal.h"
#include "qk_rows_out.cuh"
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
  int32_t n_tiles;          // tiles along N
  int32_t n_full, last_n;   // pairs: tiles of 256 columns, and columns of a product in one behind them
  int32_t y_vec;            // pairs: rows of y are whole 16-byte vectors
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
  // A product of few columns waits for the one before it on the same sums, some 125
  // cycles where its own work is 16 to 64.  So kGroup steps, each with its own sums, are
  // worked on in turns: their first 32 k, their second, and so on (16 x 8192 x 4096:
  // 11.3 us without, 9.9 with).  TMEM holds two such groups.
  constexpr int kGroup = TN <= 64 ? kQuad : 2;
  constexpr uint32_t kColumns = 2 * kGroup * TN;
  constexpr int kCols = TN / 2 < 16 ? 16 : TN / 2, kReaders = 4 * (TN / kCols);
  extern __shared__ unsigned char dynamic_smem[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 4 + 2 * kScaleSlots];
  __shared__ uint32_t tmem_at;
  __shared__ ExpertTable table;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * kStages, done0 = full0 + 16 * kStages,
                 free0 = done0 + 16, sfull0 = free0 + 16, sempty0 = sfull0 + 8 * kScaleSlots;
  const uint32_t ring = (smem_addr(dynamic_smem) + 1023u) & ~1023u;
  const uint32_t slots = ring + uint32_t(kStages * kStageBytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
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

  const int32_t tiles = table.tile0[p.experts] * p.n_tiles;  // the host bounds it
  const int32_t first = int32_t(cluster_id_x()), step = int32_t(num_clusters_x());
  const int32_t s0 = int32_t(cluster_ctarank()) * p.split_steps, s1 = min(p.groups, s0 + p.split_steps);
  struct At {
    int32_t e, n0, row0, rows;  // expert, first row of b, first row of a, rows of a
  };
  // Tile t, for t that rise: the expert is found by walking on from the last.
  auto tile = [&](int32_t t, int32_t& e) {
    while (t >= table.tile0[e + 1] * p.n_tiles) ++e;
    const int32_t in = t - table.tile0[e] * p.n_tiles, m_tiles = table.tile0[e + 1] - table.tile0[e];
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
  } else if (warp == 1) {
    // ---- products ----
    constexpr uint32_t idesc = instruction_desc_e4m3(128, TN);
    int st = 0;
    uint32_t turn = 0, it = 0;
    for (int32_t t = first; t < tiles && !failed; t += step) {
      for (int32_t s = s0; s < s1; s += kGroup, ++it) {
        const int n = min(kGroup, s1 - s);
        const uint32_t set = it & 1u;
        bool ok = wait(free0 + 8 * set, ((it >> 1) & 1u) ^ 1u);
        int last = st;
        uint32_t its_turn = turn;
        for (int q = 0; q < n && ok; ++q) {
          ok = wait(full0 + 8 * last, its_turn);
          if (++last == kStages) last = 0, its_turn ^= 1u;
        }
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        tcgen05_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kScaledStepK / 32; ++k) {
#pragma unroll
            for (int q = 0; q < kGroup; ++q) {
              if (q >= n) break;
              const int at = st + q < kStages ? st + q : st + q - kStages;
              const uint32_t sb = ring + uint32_t(at) * kStageBytes;
              mma_e4m3(tmem + (set * kGroup + q) * TN, operand_desc(sb, 0) + uint64_t(2 * k),
                       operand_desc(sb + 128 * kScaledStepK, 0) + uint64_t(2 * k), idesc, k > 0);
            }
          }
          mma_commit(done0 + 8 * set);
          for (int q = 0; q < n; ++q) mma_commit(empty0 + 8 * (st + q < kStages ? st + q : st + q - kStages));
        }
        __syncwarp();
        st = last;
        turn = its_turn;
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
        for (int g = 0; g < kQuad; g += kGroup) {
          if (q0 + g >= s1) break;
          const uint32_t set = it & 1u;
          ok = wait(done0 + 8 * set, (it >> 1) & 1u);
          if (!__all_sync(0xffffffffu, ok)) {
            failed = true;
            break;
          }
          ++it;
          tcgen05_fence_after();
          const uint32_t src = tmem + (uint32_t(quarter * 32) << 16) + set * (kGroup * TN) + uint32_t(half * kCols);
          // All of a group's sums at one trip where they fit the registers.
          constexpr int kAtOnce = kCols == 16 ? kGroup : kCols == 32 ? 2 : 1;
#pragma unroll
          for (int q1 = 0; q1 < kGroup; q1 += kAtOnce) {
            float x[kAtOnce * kCols];  // of a step that there is not: whatever TMEM holds, not used
#pragma unroll
            for (int c = 0; c < kAtOnce * kCols; c += 16)
              tmem_load_16(src + uint32_t((q1 + c / kCols) * TN + c % kCols), x + c);
#pragma unroll
            for (int c = 0; c < kAtOnce * kCols; c += 16) tmem_load_wait(x + c);
            if (q1 + kAtOnce == kGroup) {
              tcgen05_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(free0 + 8 * set);
            }
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
              const int qi = g + q1 + q;
              if (q0 + qi >= s1) break;
              const uint32_t sa = src_s + 128 * 16 + qi * (TN * 4) + half * (kCols * 4);
#pragma unroll
              for (int c = 0; c < kCols; c += 4) {
                const float4 as = ld_shared_v4(sa + c * 4);
                const float* f = x + q * kCols + c;
                const float2 both = make_float2(bs[qi], bs[qi]);  // in pairs: 3 to 5 % at 64 and 128 columns
                const float2 a0 = mul2(make_float2(as.x, as.y), both), a1 = mul2(make_float2(as.z, as.w), both);
                v[c] = fmaf(f[0], a0.x, v[c]);
                v[c + 1] = fmaf(f[1], a0.y, v[c + 1]);
                v[c + 2] = fmaf(f[2], a1.x, v[c + 2]);
                v[c + 3] = fmaf(f[3], a1.y, v[c + 3]);
              }
            }
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
      const int id = int(threadIdx.x) - 128;
      auto join = [&](auto count) {  // four neighbours of a token a thread, eight tokens at a time
        constexpr int kRanks = decltype(count)::value;
        const int32_t n = at.n0 + (id & 31) * 4;
        for (int j = int(cluster_ctarank()) + (id >> 5) * kRanks; j < at.rows; j += 8 * kRanks) {
          const uint32_t own = ring + uint32_t(j * 128 + (id & 31) * 4) * 4;
          float4 f[kRanks];
#pragma unroll
          for (int r = 0; r < kRanks; ++r) f[r] = ld_shared_cluster_v4(map_to_rank(own, uint32_t(r)));
          float sum[4] = {f[0].x, f[0].y, f[0].z, f[0].w};
#pragma unroll
          for (int r = 1; r < kRanks; ++r) sum[0] += f[r].x, sum[1] += f[r].y, sum[2] += f[r].z, sum[3] += f[r].w;
          T* y = static_cast<T*>(p.y) + int64_t(at.row0 + j) * p.N + n;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < p.N) Vec16<T>::store1(y + i, sum[i]);
        }
      };
      if (ranks == 2) join(std::integral_constant<int, 2>());
      else if (ranks == 4) join(std::integral_constant<int, 4>());
      else join(std::integral_constant<int, 8>());
    }
    __syncwarp();
    cluster_sync_all();  // the others have read this CTA's sums
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if (warp == 2) tmem_dealloc(tmem, kColumns);
}

// ---------------------------------------------------------------------------
// Tiles of 256 rows of a x 256 rows of b, a pair of CTAs each: a on TMEM's lanes,
// so a thread multiplies with one scale of a and, where b's scales are of blocks
// (!COLS), one of b: a block's sums cost a fused multiply-add each.
//
// What bounds it: the way of a block through TMEM, which holds two.  From a block's
// first product to its sums' sight 740 cycles (512 of them work), 340 to read them,
// 600 until the issuing thread knows that all 16 warps have: 1680 for two blocks,
// where the tensor cores would need 1024 (clock64 marks in one CTA, 4096 x 4864 x
// 4096).  A block in two halves of 128 columns, read and freed each by itself, takes
// longer, 543 us for 398 at 16384 x 8192 x 4096.
// Then the tiles' ends: all CTAs write 128 KB a pair at about one time, 1.7 us a tile.
// 16384 x 8192 x 4096: 396 us alone, 436 in a long run, 2520 to 2780 TFLOP/s.
// ---------------------------------------------------------------------------
// Four stages and two pieces on their way out: three stages take 443 us where these take 402
// (16384 x 8192 x 4096), five with one piece 410.
constexpr int kPairStages = 4, kPairStageBytes = 2 * 128 * kScaledStepK;  // one CTA's 128 rows of a and of b
constexpr int kPairScaleSlots = 2;
constexpr int kPairSums = 8, kPairThreads = 128 + 32 * kPairSums;  // warps that keep sums
constexpr int kPairOut = 2;  // pieces of 32 rows x 128 bytes that a warp may have on their way out
constexpr int kSplitRegistersPair = 128 * 80 + 32 * kPairSums * 208;  // what the warps' shares add up to
__host__ __device__ constexpr int pair_slot_bytes(bool cols) { return 128 * 16 + (cols ? 256 * 16 : 128); }
__host__ __device__ constexpr int pair_smem(bool cols) {  // and room to start on 1024 bytes
  return kPairStages * kPairStageBytes + kPairSums * kPairOut * kOutBytes + kPairScaleSlots * pair_slot_bytes(cols) + 1024;
}

template <bool COLS, typename T>
__global__ void __launch_bounds__(kPairThreads, 1)
    scaled_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_y, const ScaledArgs p) {
  constexpr int kStages = kPairStages, kStageBytes = kPairStageBytes, kSlots = kPairScaleSlots;
  constexpr int kSlotBytes = pair_slot_bytes(COLS), kCols = 128;
  constexpr uint32_t kColumns = 512;  // TMEM: two sets of sums
  extern __shared__ unsigned char dynamic_smem[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 2 + 2 * kSlots];
  __shared__ uint32_t tmem_at;
  __shared__ ExpertTable table;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t full0 = smem_addr(bars), done0 = full0 + 8 * kStages, free0 = done0 + 8 * kStages,
                 sfull0 = free0 + 16, sempty0 = sfull0 + 8 * kSlots;
  const uint32_t ring = (smem_addr(dynamic_smem) + 1023u) & ~1023u;  // the same in both CTAs
  const uint32_t outs = ring + uint32_t(kStages * kStageBytes), slots = outs + kPairSums * kPairOut * kOutBytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);  // the leader's producer, and the bytes of both CTAs
      // A commit: the block is summed, and the stage may be filled again.  One for both: the
      // thread that issues products is what a step of few waits for (460 -> 435 us at
      // 16384 x 8192 x 4096 with a whole warp in its loop, and less with one commit).
      mbar_init(done0 + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(free0 + 8 * i, 2 * kPairSums);  // the epilogue warps of both CTAs have read the sums
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(sfull0 + 8 * i, 2);  // this CTA's own scales
      mbar_init(sempty0 + 8 * i, kPairSums);
    }
    fence_mbar_init();
    prefetch_tensor_map(&map_a);
    prefetch_tensor_map(&map_b);
  }
  __syncwarp();
  if (warp == 2) {
    tmem_alloc_pair(smem_addr(&tmem_at), kColumns);
    tmem_relinquish_pair();
  }
  grid_dependency_wait();
  allow_dependent_launch();
  if (warp == 3) fill_table(table, p, 256, lane);
  __syncwarp();
  tcgen05_fence_before();
  cluster_sync_all();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_at;

  const int32_t tiles = table.tile0[p.experts] * p.n_tiles;  // the host bounds it
  const int32_t first = int32_t(cluster_id_x()), step = int32_t(num_clusters_x());
  struct At {
    int32_t e, n, row0, rows;  // expert, column tile, first row of a, rows of a
  };
  // Tile t, for t that rise.  Eight row tiles of an expert are walked together:
  // the pairs that run at one time share their operands in L2.
  auto tile = [&](int32_t t, int32_t& e) {
    while (t >= table.tile0[e + 1] * p.n_tiles) ++e;
    const uint32_t in = uint32_t(t - table.tile0[e] * p.n_tiles), m_tiles = uint32_t(table.tile0[e + 1] - table.tile0[e]);
    const uint32_t band = 8u * uint32_t(p.n_tiles), group = in / band, rest = in - group * band;
    const uint32_t wide = min(8u, m_tiles - group * 8u), n = rest / wide;
    At r;
    r.e = e;
    r.n = int32_t(n);
    r.row0 = table.row0[e] + int32_t(group * 8u + rest - n * wide) * 256;
    r.rows = min(256, table.row0[e + 1] - r.row0);
    return r;
  };

  bool failed = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_wait<false>(bar, parity, p.timeout_ns)) return true;
    report_status(p.status, 5);
    failed = true;
    return false;
  };

  // Registers: the launch holds 384 x 168 = 64512 (the host checks it); 128 x 80 +
  // 256 x 208 of them go to the warps that feed and to those that keep sums.
  int32_t e = 0;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0 && lane == 0) {
      // ---- producer: this CTA's half of each step's operands ----
      int64_t q = 0;
      int st = 0;
      uint32_t turn = 0;
      for (int32_t t = first; t < tiles && !failed; t += step) {
        const At at = tile(t, e);
        const int32_t a0 = at.row0 + int32_t(rank) * 128,
                      b0 = at.n * 256 + int32_t(rank) * (at.n < p.n_full ? 128 : p.last_n / 2);
        for (int32_t s = 0; s < p.groups; ++s, ++q) {
          if (!wait(done0 + 8 * st, turn ^ 1u)) break;
          const uint32_t bar = map_to_rank(full0 + 8 * st, 0), dst = ring + uint32_t(st) * kStageBytes;
          if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * st, 2 * kStageBytes);
          tma_load_3d(dst, &map_a, s * kScaledStepK, a0, 0, bar);
          tma_load_3d(dst + kStageBytes / 2, &map_b, s * kScaledStepK, b0, at.e, bar);
          if (++st == kStages) st = 0, turn ^= 1u;
        }
      }
      if (failed && rank == 0)  // leave once the loads in flight have landed: the leader's barriers count both CTAs'
        for (int64_t i = max(int64_t(0), q - kStages); i < q; ++i)
          mbar_wait<false>(full0 + 8 * uint32_t(i % kStages), uint32_t(i / kStages) & 1u, p.timeout_ns);
    } else if (warp == 1 && rank == 0) {
      // ---- products of both CTAs ----
      int st = 0;
      uint32_t turn = 0, it = 0;
      for (int32_t t = first; t < tiles && !failed; t += step) {
        const At at = tile(t, e);
        const uint32_t idesc = instruction_desc_e4m3(256, at.n < p.n_full ? 256u : uint32_t(p.last_n));
        for (int32_t s = 0; s < p.groups; ++s, ++it) {
          const uint32_t buf = it & 1u;
          const bool ok = wait(full0 + 8 * st, turn) && wait(free0 + 8 * buf, ((it >> 1) & 1u) ^ 1u);  // full long before
          if (!__all_sync(0xffffffffu, ok)) {
            failed = true;
            break;
          }
          tcgen05_fence_after();
          if (elect_one()) {
            const uint32_t sa = ring + uint32_t(st) * kStageBytes;
            const uint64_t da = operand_desc(sa, 0), db = operand_desc(sa + kStageBytes / 2, 0);
#pragma unroll
            for (int k = 0; k < kScaledStepK / 32; ++k)
              mma_e4m3_pair(tmem + buf * 256, da + uint64_t(2 * k), db + uint64_t(2 * k), idesc, k > 0);
            mma_commit_pair(done0 + 8 * st);
          }
          __syncwarp();
          if (++st == kStages) st = 0, turn ^= 1u;
        }
      }
    } else if (warp >= 2) {
      // ---- scales, four steps at a time: [128 rows of a][4], then [4][256 columns] or [2 blocks][4] ----
      const int id = (warp - 2) * 32 + lane;
      uint32_t it = 0;
      for (int32_t t = first; t < tiles && !failed; t += step) {
        const At at = tile(t, e);
        const int32_t n0 = at.n * 256, row0 = int32_t(rank) * 128;
        const float* as = p.a_scale + int64_t(at.row0) * p.groups;
        const float* bs = p.b_scale + at.e * p.b_scale_stride;
        for (int32_t s = 0; s < p.groups; s += kQuad, ++it) {
          const uint32_t slot = it % kSlots;
          const bool ok = wait(sempty0 + 8 * slot, ((it / kSlots) & 1u) ^ 1u);
          if (!__all_sync(0xffffffffu, ok)) {
            failed = true;
            break;
          }
          const uint32_t dst = slots + slot * kSlotBytes, cols = dst + 128 * 16;
          const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
          float4 f[2], g[COLS ? 4 : 1];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = row0 + id + 64 * i;
            f[i] = r < at.rows ? load_quad(as + int64_t(r) * p.groups, s, p.groups, p.scale_vec) : zero;
          }
          if constexpr (COLS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int32_t n = n0 + id + 64 * i;
              g[i] = n < p.N ? load_quad(bs + int64_t(n) * p.groups, s, p.groups, p.scale_vec) : zero;
            }
          } else {
            g[0] = id < 2 && n0 + 128 * id < p.N
                       ? load_quad(bs + int64_t(at.n * 2 + id) * p.groups, s, p.groups, p.scale_vec)
                       : zero;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) st_shared_v4(dst + (id + 64 * i) * 16, f[i]);
          if constexpr (COLS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t c = cols + (id + 64 * i) * 4;
              const float f[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
              for (int q = 0; q < kQuad; ++q) st_shared(c + q * 1024, f[q]);
            }
          } else if (id < 2) {
            st_shared_v4(cols + id * 16, g[0]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(sfull0 + 8 * slot);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- sums: half a row of the tile a thread ----
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t out_bufs = outs + uint32_t(warp - 4) * (kPairOut * kOutBytes);
    uint32_t it = 0, sit = 0, piece = 0;
    for (int32_t t = first; t < tiles && !failed; t += step) {
      const At at = tile(t, e);
      float v[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) v[j] = 0.f;
      for (int32_t s = 0; s < p.groups; s += kQuad, ++sit) {
        const uint32_t slot = sit % kSlots, src_s = slots + slot * kSlotBytes, cols = src_s + 128 * 16;
        bool ok = wait(sfull0 + 8 * slot, (sit / kSlots) & 1u);
        if (!__all_sync(0xffffffffu, ok)) {
          failed = true;
          break;
        }
        const uint32_t own = src_s + (quarter * 32 + lane) * 16;
        // Loads wait for each other, so 64 columns are asked for at a time, the second
        // 64 as the first are added: two trips to TMEM a block.  (16384 x 8192 x 4096: four
        // trips of 32 columns with the next always under way 480 us; 16 warps with four trips
        // of 16 each 500.  Single additions: packed pairs of them take 5 us more.)
        float x[COLS ? 32 : 64];
        uint32_t src = 0;
        auto summed = [&] {  // waits for the next block's sums
          const bool there = wait(done0 + 8 * (it % kStages), (it / kStages) & 1u);
          if (!__all_sync(0xffffffffu, there)) {
            failed = true;
            return false;
          }
          tcgen05_fence_after();
          src = tmem + (uint32_t(quarter * 32) << 16) + (it & 1u) * 256 + uint32_t(half * kCols);
          return true;
        };
        auto load = [&](int to, int c) {
          tmem_load_16(src + uint32_t(c), x + to);
          tmem_load_16(src + uint32_t(c + 16), x + to + 16);
        };
        auto read = [&] {  // all lanes have read their sums
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_rank(free0 + 8 * (it & 1u), 0));
          ++it;
        };
        auto add = [&](float scale, int from, int c) {  // 32 columns
#pragma unroll
          for (int j = 0; j < 32; ++j) v[c + j] = fmaf(x[from + j], scale, v[c + j]);
        };
#pragma unroll
        for (int qi = 0; qi < kQuad; ++qi) {
          if (s + qi >= p.groups || !summed()) break;
          if constexpr (COLS) {
            const float scale = ld_shared(own + qi * 4);
            // 32 columns at a time, and their scales: what is left of the registers.
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
              const uint32_t at_c = cols + uint32_t(qi * 1024 + (half * kCols + c) * 4);
              float4 bs[4];
              load(0, c);
#pragma unroll
              for (int j = 0; j < 4; ++j) bs[j] = ld_shared_v4(at_c + 16 * j);
              tmem_load_wait_32(x);
              if (c + 32 == kCols) read();
#pragma unroll
              for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float* f = x + 16 * k + 4 * j;
                  float* o = v + c + 16 * k + 4 * j;
                  // the scales' products in pairs: 601 us without at 16384 x 8192 x 4096, 566 with
                  const float2 both = make_float2(scale, scale);
                  const float2 b0 = mul2(make_float2(bs[j].x, bs[j].y), both), b1 = mul2(make_float2(bs[j].z, bs[j].w), both);
                  o[0] = fmaf(f[0], b0.x, o[0]);
                  o[1] = fmaf(f[1], b0.y, o[1]);
                  o[2] = fmaf(f[2], b1.x, o[2]);
                  o[3] = fmaf(f[3], b1.y, o[3]);
                  if (k == 0) bs[j] = ld_shared_v4(at_c + 64 + 16 * j);
                }
              }
            }
          } else {
            const float scale = ld_shared(own + qi * 4) * ld_shared(cols + half * 16 + qi * 4);
            load(0, 0);
            load(32, 32);
            tmem_load_wait_64(x);
            add(scale, 0, 0);
            load(0, 64);
            add(scale, 32, 32);
            load(32, 96);
            tmem_load_wait_64(x);
            read();
            add(scale, 0, 64);
            add(scale, 32, 96);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sempty0 + 8 * slot);
        if (failed) break;
      }
      if (failed) break;
      const int32_t r0 = int32_t(rank) * 128 + quarter * 32, j0 = at.n * 256 + half * kCols;
      const int rows_left = at.rows - r0, width = int(min(kCols, p.N - j0));  // this warp's part of y, may be <= 0
      if (width <= 0 || rows_left <= 0) continue;
      T* out = static_cast<T*>(p.y) + int64_t(at.row0 + r0) * p.N + j0;
      constexpr int E = Vec16<T>::kElems;
#pragma unroll
      for (int c = 0; c < kCols; c += 8 * E) {
        if (c >= width) break;
        uint4 u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = Vec16<T>::pack(v + c + E * k);
        // The copy from this buffer, all but one ago, has left it.
        const uint32_t buf_out = out_bufs + (piece++ % kPairOut) * kOutBytes;
        if (lane == 0) bulk_wait_read<kPairOut - 1>();
        __syncwarp();
        if (p.y_vec && rows_left >= 32) {
          // By TMA, from rows of 128 bytes in its swizzle: the warp goes on to the next
          // tile's sums while the stores of all CTAs, which come at one time, drain.
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4(buf_out + lane * 128 + ((k ^ (lane & 7)) * 16),
                         make_float4(__uint_as_float(u[k].x), __uint_as_float(u[k].y), __uint_as_float(u[k].z),
                                     __uint_as_float(u[k].w)));
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) tma_store_2d(&map_y, j0 + c, at.row0 + r0, buf_out);
        } else if (p.y_vec) {
          rows_out(buf_out, lane, u, [&](int, int r, int unit, const uint4& x) {
            const int col = c + unit * E;
            if (r < rows_left && col < width) *reinterpret_cast<uint4*>(out + int64_t(r) * p.N + col) = x;
          });
        } else {  // rows that start off 16 bytes, or end inside a vector
          elements_out<T>(buf_out, lane, u, [&](int r, int k, T x) {
            if (r < rows_left && c + k < width) out[int64_t(r) * p.N + c + k] = x;
          });
        }
        if (lane == 0) bulk_commit();  // of nothing, maybe: buffers and groups take turns alike
      }
    }
    if (lane == 0) bulk_wait();
  }
  __syncwarp();
  if (__syncthreads_or(failed)) {
    // As above: what is under way lands before this CTA's memory goes to another.
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  tcgen05_fence_before();
  cluster_sync_all();
  tcgen05_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem, kColumns);
}

// Rows of `cols` bytes that start anywhere, of two matrices, to rows of `ld` bytes
// (a multiple of 16) that start on 16: what TMA can read.  Bytes behind a row are
// whatever stands behind it, which TMA reads as zero.  A thread makes 16 bytes
// from the five words that they lie in, or from single bytes where a word would
// reach out of the matrix (1001 x 2047 x 1023 in all: 25 us, from bytes and in two launches 28).
// Sorted rows: only those between the first expert's and the last one's, and the
// weights of experts whose offsets rise, which all that have rows are among
// (one token's 8 choices of 64 experts, 4096 x 4095: 89 us, with all weights 422).
// What a tile reads beyond them ends in rows that it does not store.
struct PadArgs {
  const uint8_t* in[2];  // b, a
  uint8_t* out[2];
  int64_t rows[2];         // 0: this one is read where it is
  int64_t M;               // what offsets lie within
  const int32_t* offsets;  // [experts + 1], null: all rows
  int32_t experts;
  int32_t expert_rows;     // rows of b of one expert
  int32_t cols, ld;
};
__global__ void __launch_bounds__(256) pad_rows_kernel(const PadArgs a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  auto offset = [&](int32_t e) { return min(max(int64_t(a.offsets[e]), int64_t(0)), a.M); };
  int64_t end = -1;  // of the last expert's rows: the largest offset, found by the first row of a
  for (int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); r < a.rows[0] + a.rows[1]; r += int64_t(gridDim.x) * 8) {
    const int which = r >= a.rows[0];
    const int64_t row = which ? r - a.rows[0] : r;
    if (a.offsets != nullptr) {
      if (which) {
        if (end < 0) {
          int32_t top = 0;
          for (int32_t e = lane; e <= a.experts; e += 32) top = max(top, int32_t(offset(e)));
          end = __reduce_max_sync(0xffffffffu, top);
        }
        if (row < offset(0) || row >= end) continue;
      } else {
        const int32_t e = int32_t(row / a.expert_rows);
        if (offset(e + 1) <= offset(e)) continue;
      }
    }
    const uint8_t* in = a.in[which];
    const uintptr_t lo = reinterpret_cast<uintptr_t>(in), hi = lo + uintptr_t(a.rows[which]) * uintptr_t(a.cols);
    uint8_t* dst = a.out[which] + row * a.ld;
    for (int32_t c = lane * 16; c < a.cols; c += 512) {
      const uintptr_t s = lo + uintptr_t(row) * uintptr_t(a.cols) + uintptr_t(c), s4 = s & ~uintptr_t(3);
      uint32_t w[5];
      if (s4 >= lo && s4 + 20 <= hi) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = reinterpret_cast<const uint32_t*>(s4)[i];
        const uint32_t shift = uint32_t(s & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], shift);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (s + 4 * i + b < hi) w[i] |= uint32_t(*reinterpret_cast<const uint8_t*>(s + 4 * i + b)) << (8 * b);
        }
      }
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace qk
