// qk_product_kernel.cuh -- matrix products on tcgen05 with the epilogues of the
// linear cross-entropy (sm_103a).
//
//   C[i,j] = sum_k A(i,k) B(j,k),  bf16 operands, fp32 sums
//
// What bounds it: the tensor cores.  A pair of CTAs forms a 256 x 256 tile; a
// step of 64 k is 4 products of 16 k and 64 KB of operands through TMA, so each
// byte that reaches shared memory is used 128 times.  Warp 0 keeps TMA loads
// six steps ahead, warp 1 of the leading CTA issues the products, warps 4-11
// take finished sums out of TMEM (which holds two sets) and turn them into
// outputs while the next ones are formed.  The grid is persistent: one CTA an SM.
//
// The tensor core adds to a sum by cutting off what does not fit, always toward
// zero: a chain of n products of 16 k is short by about n 2^-25.5 of itself (a
// sum over 8192 k measured 1e-5 off, where rounding to nearest gives 1e-6).  So
// a chain ends after `chunk` steps of 64 k, and the chains of a tile are added in
// registers, to nearest.  16 steps for bf16 (lse 2.6e-7 off at K = 4096), whose
// outputs of consequence are bf16; 2 (48 products) for float32, whose gradients
// are 4e-7 off, against 0.8 to 1.6e-6 of fp32 products (with 1 step 2e-7, for
// 5 to 10 % more time).
// Shorter chains cost time and power.  8192 x 131072 x 4096 forward in a long
// run: 16 steps 5.22 ms (lse 2.6e-7 off), 12 5.31 (1.9e-7), 8 5.41 (1.3e-7), 4
// 5.77 (7e-8); float32 products with sums to nearest are 1e-7 off.  The bf16
// backward of 8192 x 32000 x 4096: 4.06 ms with 16 steps, 4.21 with 8.
//
// An operand is stored with k innermost (K-major) or with its rows innermost
// (MN-major): h, w and g serve as either, without a transposed copy.
//
// float32 operands come as three bf16 planes, x = x0 + x1 + x2 with 8 bits of
// the significand each (what is left is below 2^-26 of x); the products x_a y_b
// with a + b <= 2 are summed, the small ones first.  What is left out is below
// 2^-25 of a term.  A step loads its six operand tiles once for its six plane
// pairs, half the bytes of two tiles for each: what steps of one pair wait for is
// the way from L2 to the SMs (0.34 to 0.38 us for 64 KB a pair of CTAs, whatever
// they multiply).  4096 x 16384 x 1024 backward: 1474 us, 1679 TFLOP/s of bf16 products.
#pragma once

#include "qk_internal.h"
#include "qk_tensor.cuh"

namespace qk {

constexpr int kProductThreads = 384;  // 4 warps that feed the tensor cores, 8 for the sums
constexpr int kTileM = 256;       // rows of a pair's tile
constexpr int kTileN = 256;       // columns of one, where there are enough
constexpr int kStepK = 64;        // k of one pipeline step: 128 bytes
constexpr int kABytes = 128 * kStepK * 2;  // one CTA's part of a step of A
constexpr int kSplitRegisters = 128 * 64 + 256 * 216;  // what the warps' shares add up to
constexpr int kOutBytes = 32 * 128;        // an epilogue warp's 32 rows of 128 bytes on their way out

// kEpiLseCols: C's columns are the tokens (few), its rows the vocabulary.
// kEpiFinish: the last addition to fp32 sums, rounded to the output.
enum Epilogue : int { kEpiLse = 0, kEpiGrad = 1, kEpiAccum = 2, kEpiStore = 3, kEpiLseCols = 4, kEpiFinish = 5 };

// Shared memory by the tile's columns TN: six stages of 32 KB, or ten of A's
// 16 KB and B's TN / 2 rows when that is little, and the way out.
// Three planes at once take two stages of 96 KB.
__host__ __device__ constexpr int product_stages(int tn, int planes) { return planes == 3 ? 2 : tn == kTileN ? 6 : 10; }
__host__ __device__ constexpr int product_stage_bytes(int tn, int planes) {
  return planes * (kABytes + tn / 2 * kStepK * 2);
}
__host__ __device__ constexpr int product_smem(int tn, int planes) {  // and room to start on 1024 bytes
  return product_stages(tn, planes) * product_stage_bytes(tn, planes) + (tn == kTileN ? 8 * kOutBytes : 0) + 1024;
}

struct XentRow {   // what the gradient needs of a row
  float lse, g, zf;  // g: dloss / scale (NaN for a bad target); zf = 1 + 2 z lse
  int32_t target;    // -1: none, -2: an ignored row
};

struct ProductArgs {
  int32_t rows, cols;        // of C
  int32_t steps;             // steps of 64 k
  int32_t depth;             // k
  int32_t m_tiles, n_tiles;
  int32_t n_full, last_n;    // column tiles of TN columns (the first ones); columns of a product in the last
  int32_t chunk;             // steps of one chain of products
  int32_t splits, split_steps;  // the k axis in pieces of split_steps steps
  uint64_t timeout_ns;
  int* status;
  // epilogues; v0: vocabulary index of column 0
  int64_t v0;
  const int64_t* targets;    // lse
  float2* part;              // lse: [half column tile, or CTA][part_ld] (maximum, sum)
  int64_t part_ld;
  int64_t part0;             // lse over columns: first pair's place in the list
  float* at_target;          // lse: logit of the target
  const XentRow* row;        // grad
  void* out;                 // grad: bf16 [planes][rows][ld]; accum: fp32 [splits][rows][ld]; store: [rows][ld]
  int64_t ld, plane_stride;  // elements
  int32_t first;             // accum: overwrite
  const float* sum;          // finish: fp32 [rows][sum_ld]
  int64_t sum_ld;
  int32_t vec;               // store: rows start on 16 bytes
  const float* scale;        // accum, store, finish: factor (device)
};

// Splits a float into three bf16 parts; what is not finite stays in the first.
__device__ __forceinline__ void split3(float x, __nv_bfloat16* b) {
  b[0] = __float2bfloat16_rn(x);
  const float r1 = x - __bfloat162float(b[0]);
  const bool fin = fabsf(x) < __int_as_float(0x7f800000) && fabsf(r1) < __int_as_float(0x7f800000);
  b[1] = __float2bfloat16_rn(fin ? r1 : 0.f);
  b[2] = __float2bfloat16_rn(fin ? r1 - __bfloat162float(b[1]) : 0.f);
}

// 32 rows of 128 bytes from "a row a lane" (u[0..7], 16 bytes each) to memory:
// put(k, row, unit, x) gets each 16 bytes once (k: 0..7, row = 4 k + lane / 8), eight lanes on the 128 bytes of one
// row, so that stores are whole lines.  A lane storing its own row's vectors
// touches 32 lines an instruction: dh at 8192 x 32000 x 4096 ran at 1150 TFLOP/s
// that way.  Units are XORed with the row: no bank is hit twice.
template <typename F>
__device__ __forceinline__ void rows_out(uint32_t buf, int lane, const uint4* u, F put) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((k ^ (lane & 7)) * 16)),
                 "r"(u[k].x), "r"(u[k].y), "r"(u[k].z), "r"(u[k].w)
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int row = k * 4 + (lane >> 3), unit = lane & 7;
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(buf + row * 128 + ((unit ^ (row & 7)) * 16))
                 : "memory");
    put(k, row, unit, x);
  }
  __syncwarp();
}

// The same for rows that start off 16 bytes: put(row, column, x) gets single
// elements, a warp's lanes on consecutive columns of one row.
template <typename T, typename F>
__device__ __forceinline__ void elements_out(uint32_t buf, int lane, const uint4* u, F put) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((k ^ (lane & 7)) * 16)),
                 "r"(u[k].x), "r"(u[k].y), "r"(u[k].z), "r"(u[k].w)
                 : "memory");
  __syncwarp();
#pragma unroll 8
  for (int row = 0; row < 32; ++row) {
#pragma unroll
    for (int col = lane; col < int(128 / sizeof(T)); col += 32) {
      const uint32_t byte = uint32_t(col) * sizeof(T);
      const uint32_t at = buf + row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15u);
      if constexpr (sizeof(T) == 4) {
        float x;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
        put(row, col, x);
      } else {
        uint16_t x;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
        put(row, col, __ushort_as_bfloat16(x));
      }
    }
  }
  __syncwarp();
}

// Tile number -> (split, row tile, column tile).  Eight row tiles are walked
// together: the pairs that run at one time then share their operands in L2
// (76 pairs: 8 row tiles x 9.5 column tiles, a quarter of the loads unique).
// A last column tile of fewer columns comes after all others, as a narrower
// product: what is short goes where the last wave has room.
// 32-bit: the host refuses more tiles (64-bit divisions cost a thousand cycles
// a tile, which shows where a tile is a step or two).
struct TileAt {
  int split, m, n;
};
__device__ __forceinline__ TileAt tile_at(const ProductArgs& p, uint32_t t) {
  TileAt r;
  const uint32_t full = uint32_t(p.n_full), per = uint32_t(p.m_tiles) * full, all = per * uint32_t(p.splits);
  if (t >= all) {
    const uint32_t in = t - all;
    r.split = int(in / uint32_t(p.m_tiles));
    r.m = int(in - uint32_t(r.split) * uint32_t(p.m_tiles));
    r.n = int(full);
    return r;
  }
  r.split = p.splits == 1 ? 0 : int(t / per);
  const uint32_t in = t - uint32_t(r.split) * per, band = 8u * full, group = in / band, rest = in - group * band;
  const uint32_t wide = min(8u, uint32_t(p.m_tiles) - group * 8u);
  r.n = int(rest / wide);
  r.m = int(group * 8u + rest - uint32_t(r.n) * wide);
  return r;
}

template <int EPI, bool A_MN, bool B_MN, typename T, int TN, int PLANES>
__global__ void __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const ProductArgs p) {
  constexpr int kStages = product_stages(TN, PLANES), kStageBytes = product_stage_bytes(TN, PLANES);
  constexpr int kBBytes = TN / 2 * kStepK * 2;  // one CTA's part of a step of B
  static_assert(PLANES == 1 || TN == kTileN, "three planes at once: full tiles");
  // A product of few columns waits for the one before it on the same sums, some
  // 125 cycles where its own work is 16 to 64; so a step's products of 16 k go to
  // four sets of sums (two at 128 columns), which the epilogue adds.  Tiles of TN
  // columns below 256 do so always, g's product in a narrow last column tile.
  constexpr int kParts = TN == kTileN ? 1 : 4, kSet = kParts * TN;
  constexpr uint32_t kColumns = 2 * kSet;  // TMEM: two sets of sums, or of four times them
  static_assert(!B_MN || TN == kTileN, "MN-major B comes in boxes of 64 columns");
  extern __shared__ unsigned char dynamic_smem[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
  __shared__ uint32_t tmem_at;
  __shared__ float2 joint[EPI == kEpiLseCols ? 4 : 1][EPI == kEpiLseCols ? TN : 1];

  // Columns of an epilogue thread, and the warps that take part.
  constexpr int kCols = TN / 2 < 16 ? 16 : TN / 2, kReaders = 4 * (TN / kCols);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * kStages, done0 = full0 + 16 * kStages,
                 free0 = done0 + 16;
  const uint32_t ring = (smem_addr(dynamic_smem) + 1023u) & ~1023u;  // the same in both CTAs
  const uint32_t tiles = uint32_t(p.m_tiles) * uint32_t(p.n_tiles) * uint32_t(p.splits);
  const uint32_t first_tile = cluster_id_x(), tile_step = num_clusters_x();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);   // the leader's producer, and the bytes of both CTAs
      mbar_init(empty0 + 8 * s, 1);  // a commit of the leader's products
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(done0 + 8 * i, 1);   // a commit: the chain is summed
      mbar_init(free0 + 8 * i, 2 * kReaders);  // the epilogue warps of both CTAs have read it
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
  tcgen05_fence_before();
  cluster_sync_all();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_at;
  grid_dependency_wait();
  allow_dependent_launch();

  auto parts_of = [&](int n) {
    // Only g's product: a narrow tile of dw or dh waits for A's steps all the
    // same (2047 x 8191 x 513 fp32: 148 us without, 151 with), and the forward's
    // loop is 3 % slower with the choice in it.
    if (TN < kTileN || EPI != kEpiGrad || PLANES == 3) return kParts;
    return n < p.n_full || p.last_n > 128 ? 1 : p.last_n > 64 ? 2 : 4;
  };
  bool failed = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (mbar_wait<false>(bar, parity, p.timeout_ns)) return true;
    report_status(p.status, 5);
    failed = true;
    return false;
  };

  // Registers: the launch holds 384 x 168 = 64512 (the host checks it); 128 x 64
  // + 256 x 216 = 63488 of them go to the warps that feed and to those that keep sums.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0 && lane == 0) {
      // ---- producer: this CTA's half of each step's operands ----
      constexpr int half_n = TN / 2;
      constexpr uint32_t bytes = 2u * uint32_t(kStageBytes);
      int64_t q = 0;  // steps issued
      int st = 0;
      uint32_t turn = 0;
      for (uint32_t t = first_tile; t < tiles && !failed; t += tile_step) {
        const TileAt at = tile_at(p, t);
        const int a0 = at.m * kTileM + int(rank) * 128, b0 = at.n * TN + int(rank) * (at.n < p.n_full ? half_n : p.last_n / 2);
        const int s0 = at.split * p.split_steps, s1 = min(p.steps, s0 + p.split_steps);
        for (int s = s0; s < s1; ++s, ++q) {
          if (!wait(empty0 + 8 * st, turn ^ 1u)) break;
          const int k = s * kStepK;
          const uint32_t bar = map_to_rank(full0 + 8 * st, 0);
          if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * st, bytes);
          const uint32_t sa = ring + uint32_t(st) * kStageBytes, sb = sa + PLANES * kABytes;
#pragma unroll
          for (int pl = 0; pl < PLANES; ++pl) {
            const uint32_t da = sa + pl * kABytes, db = sb + pl * kBBytes;
            if constexpr (A_MN) {
              tma_load_3d(da, &map_a, a0, k, pl, bar);
              tma_load_3d(da + kABytes / 2, &map_a, a0 + 64, k, pl, bar);
            } else {
              tma_load_3d(da, &map_a, k, a0, pl, bar);
            }
            if constexpr (B_MN) {
              for (int i = 0; i < half_n / 64; ++i)
                tma_load_3d(db + uint32_t(i) * (64 * kStepK * 2), &map_b, b0 + 64 * i, k, pl, bar);
            } else {
              tma_load_3d(db, &map_b, k, b0, pl, bar);
            }
          }
          if (++st == kStages) st = 0, turn ^= 1u;
        }
      }
      // A failed launch leaves once the loads in flight have landed: the leader's
      // barriers count those of both CTAs.
      if (failed && rank == 0)
        for (int64_t i = max(int64_t(0), q - kStages); i < q; ++i)
          mbar_wait<false>(full0 + 8 * uint32_t(i % kStages), uint32_t(i / kStages) & 1u, p.timeout_ns);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---- products of both CTAs ----
      constexpr uint32_t kLbo = 64 * kStepK * 2;                       // MN-major: the next 64 rows
      constexpr uint32_t kAStep = (A_MN ? 16 * 128 : 32) >> 4, kBStep = (B_MN ? 16 * 128 : 32) >> 4;  // 16 k
      const int tail_parts = (p.depth - (p.steps - 1) * kStepK + 15) / 16;
      int st = 0;
      uint32_t turn = 0, it = 0;  // it: chains begun
      for (uint32_t t = first_tile; t < tiles && !failed; t += tile_step) {
        const TileAt at = tile_at(p, t);
        const int s0 = at.split * p.split_steps, s1 = min(p.steps, s0 + p.split_steps);
        const uint32_t idesc = instruction_desc(A_MN, B_MN, at.n < p.n_full ? uint32_t(TN) : uint32_t(p.last_n));
        const int parts = parts_of(at.n);
        const uint32_t stride = uint32_t(kSet / parts);
        for (int c0 = s0; c0 < s1 && !failed; c0 += p.chunk, ++it) {
          const uint32_t acc = it & 1u;
          if (!wait(free0 + 8 * acc, ((it >> 1) & 1u) ^ 1u)) break;
          tcgen05_fence_after();
          const uint32_t d = tmem + acc * kSet;
          const int c1 = min(s1, c0 + p.chunk);
          for (int s = c0; s < c1; ++s) {
            if (!wait(full0 + 8 * st, turn)) break;
            tcgen05_fence_after();
            const uint32_t sa = ring + uint32_t(st) * kStageBytes;
            const uint64_t da = operand_desc(sa, A_MN ? kLbo : 0);
            const uint64_t db = operand_desc(sa + PLANES * kABytes, B_MN ? kLbo : 0);
            const bool tail = s == p.steps - 1;  // the last step may hold fewer k
            if constexpr (PLANES == 3) {  // the six plane pairs of these k, the small ones first
              const int count = tail ? tail_parts : kStepK / 16;
              bool add = s > c0;
#pragma unroll
              for (int pair = 0; pair < 6; ++pair) {
                const int pa = pair < 3 ? 2 - pair : pair == 3 ? 1 : 0, pb = pair < 3 ? pair : pair == 4 ? 1 : 0;
                for (int k = 0; k < count; ++k) {
                  mma_bf16_pair(d, da + uint64_t(pa * (kABytes >> 4) + k * kAStep),
                                db + uint64_t(pb * (kBBytes >> 4) + k * kBStep), idesc, add);
                  add = true;
                }
              }
            } else if (parts == 1 && tail && tail_parts < kStepK / 16) {
              for (int k = 0; k < tail_parts; ++k)
                mma_bf16_pair(d, da + uint64_t(k) * kAStep, db + uint64_t(k) * kBStep, idesc, s > c0 || k > 0);
            } else {
#pragma unroll
              for (int k = 0; k < kStepK / 16; ++k)
                mma_bf16_pair(d + uint32_t(k & (parts - 1)) * stride, da + uint64_t(k) * kAStep,
                              db + uint64_t(k) * kBStep, idesc, s > c0 || k >= parts);
            }
            mma_commit_pair(empty0 + 8 * st);
            if (++st == kStages) st = 0, turn ^= 1u;
          }
          if (!failed) mma_commit_pair(done0 + 8 * acc);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- epilogue: half a row of the tile a thread ----
    const int quarter = warp & 3, half = (warp - 4) >> 2;  // TMEM lanes of a warp: 32 (warp % 4) and up
    const uint32_t buf = ring + uint32_t(kStages * kStageBytes) + uint32_t(warp - 4) * kOutBytes;
    // kEpiLseCols: each lane's running (maximum, sum) of its tokens over the
    // vocabulary rows it meets, joined over the lanes once at the end.
    float run_m[EPI == kEpiLseCols ? kCols : 1], run_s[EPI == kEpiLseCols ? kCols : 1];
    int run_t[EPI == kEpiLseCols ? kCols : 1];
    if constexpr (EPI == kEpiLseCols) {
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int token = half * kCols + j;
        run_m[j] = kNegInf;
        run_s[j] = 0.f;
        const int64_t tg = token < p.cols ? p.targets[token] : -1;
        run_t[j] = tg >= p.v0 && tg < p.v0 + p.rows ? int(tg - p.v0) : -1;
      }
    }
    float factor = 1.f;
    if constexpr (EPI == kEpiAccum || EPI == kEpiStore || EPI == kEpiFinish) factor = *p.scale;
    uint32_t it = 0;
    for (uint32_t t = first_tile; t < tiles && !failed && half * kCols < TN; t += tile_step) {
      const TileAt at = tile_at(p, t);
      const int s0 = at.split * p.split_steps, s1 = min(p.steps, s0 + p.split_steps);
      const int64_t i = int64_t(at.m) * kTileM + rank * 128 + quarter * 32 + lane;
      const int64_t j0 = int64_t(at.n) * TN + half * kCols;
      const bool live = i < p.rows;
      const int rows_left = int(min(int64_t(32), p.rows - (i - lane)));  // this warp's rows of C, may be <= 0
      const int width = int(min(int64_t(kCols), p.cols - j0));  // this half's columns of C, may be <= 0

      // What the outputs need of the row, asked for while the sums are formed.
      XentRow row = {0.f, 0.f, 0.f, -2};
      int64_t row_target = -1;
      if constexpr (EPI == kEpiGrad) {
        if (live) row = p.row[i];
      }
      if constexpr (EPI == kEpiLse) {
        if (live) row_target = p.targets[i];
      }

      float v[kCols];
      for (int c0 = s0; c0 < s1; c0 += p.chunk, ++it) {
        const uint32_t acc = it & 1u;
        const bool summed = wait(done0 + 8 * acc, (it >> 1) & 1u);
        if (!__all_sync(0xffffffffu, summed)) {  // a warp gives up as one: its lanes meet again below
          failed = true;
          break;
        }
        tcgen05_fence_after();
        const uint32_t src = tmem + (uint32_t(quarter * 32) << 16) + acc * kSet + uint32_t(half * kCols);
        __syncwarp();  // the loads are the warp's
        if constexpr (kParts > 1) {
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            float x[kParts][16];
#pragma unroll
            for (int k = 0; k < kParts; ++k) tmem_load_16(src + uint32_t(k * TN + c), x[k]);
#pragma unroll
            for (int k = 0; k < kParts; ++k) tmem_load_wait(x[k]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float sum = (x[0][j] + x[1][j]) + (x[2][j] + x[3][j]);
              v[c + j] = c0 == s0 ? sum : v[c + j] + sum;
            }
          }
        } else if (c0 == s0) {
#pragma unroll
          for (int c = 0; c < kCols; c += 16) tmem_load_16(src + uint32_t(c), v + c);
#pragma unroll
          for (int c = 0; c < kCols; c += 16) tmem_load_wait(v + c);
        } else {
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            float x[16];
            tmem_load_16(src + uint32_t(c), x);
            tmem_load_wait(x);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[c + j] += x[j];
          }
        }
        if (const int parts = parts_of(at.n); EPI == kEpiGrad && parts > 1 && half == 0) {
          const int stride = kTileN / parts;  // all the columns of such a tile are this half's
          for (int k = 1; k < parts; ++k) {
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
              if (c >= stride) continue;
              float x[16];
              tmem_load_16(src + uint32_t(k * stride + c), x);
              tmem_load_wait(x);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[c + j] += x[j];
            }
          }
        }
        tcgen05_fence_before();
        __syncwarp();  // all lanes have read their sums
        if (lane == 0) mbar_arrive_cluster(map_to_rank(free0 + 8 * acc, 0));
      }
      if (failed) break;

      if constexpr (EPI == kEpiLseCols) {
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          if (run_t[j] == int(i)) p.at_target[half * kCols + j] = v[j];
          const float mn = fmaxf(run_m[j], v[j]);
          // All -inf so far: shift by 0, so that a NaN still shows.
          const float base = mn == kNegInf ? 0.f : mn * kLog2e;
          run_s[j] = (run_m[j] == kNegInf ? run_s[j] : run_s[j] * exp2_approx(fmaf(run_m[j], kLog2e, -base))) +
                     exp2_approx(fmaf(v[j], kLog2e, -base));
          run_m[j] = mn;
        }
      } else if constexpr (EPI == kEpiLse) {
        // (maximum, sum of exponentials) of the half row; columns past the last count as -inf
        if (!live) continue;
        const int64_t target = row_target >= 0 ? row_target - p.v0 - j0 : -1;  // any int64 may stand there
        if (target >= 0 && target < width) {
          float x = 0.f;
#pragma unroll
          for (int j = 0; j < kCols; ++j)  // as PTX: in C++ it becomes an indexed load, and v leaves the registers
            asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %2, %3;\n\t@p mov.f32 %0, %1;\n\t}"
                : "+f"(x)
                : "f"(v[j]), "r"(int(target)), "r"(j));
          p.at_target[i] = x;
        }
        float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf}, sum[4] = {};
        if (width < kCols) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] = j < width ? v[j] : kNegInf;
        }
#pragma unroll
        for (int j = 0; j < kCols; ++j) mx[j & 3] = fmaxf(mx[j & 3], v[j]);
        const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // All -inf: shift by 0, so that a NaN among them still shows.
        const float base = m == kNegInf ? 0.f : m * kLog2e;
#pragma unroll
        for (int j = 0; j < kCols; ++j) sum[j & 3] += exp2_approx(fmaf(v[j], kLog2e, -base));
        p.part[(2 * (p.v0 / TN + at.n) + half) * p.part_ld + i] =
            make_float2(m, (sum[0] + sum[1]) + (sum[2] + sum[3]));
      } else if constexpr (EPI == kEpiGrad) {
        if (width <= 0) continue;
        const int64_t at_t = row.target >= 0 ? row.target - p.v0 - j0 : -1;
        const int target = at_t >= 0 && at_t < width ? int(at_t) : -1;
        // g = dloss (zf exp(x - lse) - onehot): three operations a column, and the
        // one-hot's only in a warp that holds a target here.
        const float f = row.zf * row.g, lb = -row.lse * kLog2e;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          // bf16: one fused step (lse log2(e) is rounded, 2^-20 of p); float32 subtracts first
          const float e = sizeof(T) == 2 ? fmaf(v[j], kLog2e, lb) : (v[j] - row.lse) * kLog2e;
          v[j] = exp2_approx(e) * f;
        }
        if (__any_sync(0xffffffffu, target >= 0)) {
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            if (j == target) v[j] -= row.g;
        }
        if (row.target == -2) {  // ignored: zero, whatever its logits are
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] = 0.f;
        }
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (i - lane) * p.ld + j0;
#pragma unroll
        for (int c = 0; c < kCols; c += 64) {  // ld is a multiple of 8: whole vectors stay inside the row
          if (c >= width) break;
#pragma unroll
          for (int pl = 0; pl < (sizeof(T) == 2 ? 1 : 3); ++pl) {
            uint4 u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              u[k] = Vec16<__nv_bfloat16>::pack(v + c + 8 * k);
              if constexpr (sizeof(T) == 4) {  // the next plane holds what this one left
                float f[8];
                Vec16<__nv_bfloat16>::unpack(u[k], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c + 8 * k + e] -= f[e];
              }
            }
            rows_out(buf, lane, u, [&](int, int r, int unit, const uint4& x) {
              const int col = c + unit * 8;
              if (r < rows_left && col < width)
                *reinterpret_cast<uint4*>(out + pl * p.plane_stride + r * p.ld + col) = x;
            });
          }
        }
      } else if constexpr (EPI == kEpiAccum) {
        if (width <= 0) continue;
#pragma unroll
        for (int j = 0; j < kCols; ++j) v[j] *= factor;
        float* out = static_cast<float*>(p.out) + (int64_t(at.split) * p.rows + (i - lane)) * p.ld + j0;
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          if (c >= width) break;
          uint4 u[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] = Vec16<float>::pack(v + c + 4 * k);
          rows_out(buf, lane, u, [&](int, int r, int unit, const uint4& x) {
            const int col = c + unit * 4;
            if (r >= rows_left || col >= width) return;  // ld is a multiple of 4
            float* o = out + r * p.ld + col;
            // Later pieces add at L2, which spares the loads: this launch is the
            // only adder of an element, so the bits do not depend on any order.
            if (p.first) {
              *reinterpret_cast<uint4*>(o) = x;
            } else {
              asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(o),
                           "f"(__uint_as_float(x.x)), "f"(__uint_as_float(x.y)), "f"(__uint_as_float(x.z)),
                           "f"(__uint_as_float(x.w))
                           : "memory");
            }
          });
        }
      } else if constexpr (EPI == kEpiFinish) {
        if (width <= 0) continue;
#pragma unroll
        for (int j = 0; j < kCols; ++j) v[j] *= factor;
        const float* sum = p.sum + (i - lane) * p.sum_ld + j0;
        T* out = static_cast<T*>(p.out) + (i - lane) * p.ld + j0;
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          if (c >= width) break;
          uint4 u[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] = Vec16<float>::pack(v + c + 4 * k);
          // The sums so far, all eight loads before the first store: one after the
          // other they cost a trip to memory each.
          float4 y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = k * 4 + (lane >> 3), col = c + (lane & 7) * 4;
            if (r < rows_left && col < width) y[k] = *reinterpret_cast<const float4*>(sum + r * p.sum_ld + col);
          }
          rows_out(buf, lane, u, [&](int k, int r, int unit, const uint4& x) {
            const int col = c + unit * 4;
            if (r >= rows_left || col >= width) return;  // sum_ld is a multiple of 4
            float f[4];
            Vec16<float>::unpack(x, f);
            f[0] += y[k].x, f[1] += y[k].y, f[2] += y[k].z, f[3] += y[k].w;
            T* o = out + r * p.ld + col;
            if (p.vec) {
              if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint2*>(o) = make_uint2(Vec16<T>::pack2(f[0], f[1]), Vec16<T>::pack2(f[2], f[3]));
              } else {
                *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (col + e < width) Vec16<T>::store1(o + e, f[e]);
            }
          });
        }
      } else {
        if (width <= 0) continue;
        T* out = static_cast<T*>(p.out) + (i - lane) * p.ld + j0;
        constexpr int E = Vec16<T>::kElems;
#pragma unroll
        for (int j = 0; j < kCols; ++j) v[j] *= factor;
#pragma unroll
        for (int c = 0; c < kCols; c += 8 * E) {
          if (c >= width) break;
          uint4 u[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] = Vec16<T>::pack(v + c + E * k);
          if (p.vec) {
            rows_out(buf, lane, u, [&](int, int r, int unit, const uint4& x) {
              const int col = c + unit * E;
              if (r < rows_left && col < width) *reinterpret_cast<uint4*>(out + r * p.ld + col) = x;
            });
          } else {  // rows that start off 16 bytes, or end inside a vector
            elements_out<T>(buf, lane, u, [&](int r, int k, T x) {
              if (r < rows_left && c + k < width) out[r * p.ld + c + k] = x;
            });
          }
        }
      }
    }
    if constexpr (EPI == kEpiLseCols) {
      // One pair a CTA and token: the lanes of each warp, then the four warps in order.
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const float m = group_max<32>(run_m[j]);
        const float s = group_sum<32>(run_m[j] == kNegInf ? run_s[j] : run_s[j] * exp2_approx((run_m[j] - m) * kLog2e));
        if (lane == 0 && half * kCols < TN) joint[quarter][half * kCols + j] = make_float2(m, s);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the eight epilogue warps
      const int token = int(threadIdx.x) - 128;
      if (token < p.cols) {
        float m = kNegInf, s = 0.f;
        for (int k = 0; k < 4; ++k) m = fmaxf(m, joint[k][token].x);
        for (int k = 0; k < 4; ++k) {
          const float2 b = joint[k][token];
          s += b.x == kNegInf ? b.y : b.y * exp2_approx((b.x - m) * kLog2e);
        }
        p.part[((p.part0 + first_tile) * 2 + rank) * p.part_ld + token] = make_float2(m, s);
      }
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
  if (warp == 2) tmem_dealloc_pair(tmem, kColumns);
}

}  // namespace qk
