// qk_few_tokens.cuh -- the float32 linear cross-entropy of up to 32 tokens on the
// fp32 units (sm_103a).
//
// The bf16 planes that the products of qk_product_kernel.cuh want move 12 bytes
// more for each 4-byte weight and pass; here w is read once (and dw written).
// 80000 x 464, by planes and so: forward of 4 to 32 tokens 142 to 156 us, and 32
// (4 tokens), 55 (16) or 104 (32), where w's bytes take 22; backward 272 to 279,
// and 99, 181 or 309 (where they take 67, read twice and written).
// What bounds it: w's bytes at 4 tokens.  At 16 and 32 tokens not yet the
// multiplications, which run at 22 TFLOP/s, a quarter to a third of the fp32
// units' rate: at 32 a 16-byte read of h from shared memory feeds only 8 of them
// (R = 2 rows), at 16 no load of w is under way while one is multiplied.
// (bf16 rows that have to be copied are faster by the products from 4 tokens on:
// one copy, and a quarter of the bytes.)
#pragma once

#include "qk_product_kernel.cuh"  // XentRow

namespace qk {

constexpr int kFewLogitThreads = 512;  // one CTA an SM, beside h in its shared memory
constexpr int kFewThreads = 256;

struct FewArgs {
  const void* h;  // [M, K]
  const void* w;  // [V, K]
  int64_t V;
  int32_t M, K;
  // forward
  const int64_t* targets;
  float2* part;      // [CTA][M] (maximum, sum)
  float* at_target;  // [M]
  // backward
  const XentRow* row;
  float* g;          // [V][MT]
  float* sum;        // [splits][M][ld] fp32 sums of dh, or null
  void* dw;          // [V, K] or null
  const float* scale;
  int64_t ld;
  int32_t chunk;     // k of h in shared memory at a time
  int32_t columns;   // threads of a CTA along k: 64, 128 or 256
  int64_t per_split; // vocabulary rows of a split
};

// N values a lane, each to be summed over the warp: after the exchange lane l
// holds the sums of values l N/32 ... (l + 1) N/32 - 1 in x[0 .. N/32), with
// N - N/32 shuffles instead of 5 N.
template <int N>
__device__ __forceinline__ void warp_transpose_sum(float* x, int lane) {
#pragma unroll
  for (int o = 16, n = N / 2; o > 0; o >>= 1, n >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = upper ? x[i + n] : x[i], send = upper ? x[i] : x[i + n];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
}

// Logits of R vocabulary rows and MT tokens a warp at a time, h in shared memory
// (all of it, or `chunk` k of it for each round of rows), lanes along k.
// Forward: running (maximum, sum) of each token, one pair a CTA.  GRAD: g
// instead.  KV: k of a load (4 where rows are aligned).
template <typename T, int MT, int KV, bool GRAD>
__global__ void __launch_bounds__(kFewLogitThreads, 1) few_logits_kernel(const FewArgs a) {
  constexpr int R = 64 / MT > 8 ? 8 : 64 / MT, N = R * MT, PER = N / 32, NW = kFewLogitThreads / 32;
  static_assert(N % 32 == 0, "whole values a lane");
  extern __shared__ __align__(16) float hs[];  // [MT][chunk]
  __shared__ float2 joint[GRAD ? 1 : NW][GRAD ? 1 : N];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = a.K, KC = a.chunk;
  auto stage = [&](int64_t k0) {  // h's columns [k0, k0 + KC)
    const int left = int(min(int64_t(KC), K - k0));
    for (int m = warp; m < MT; m += NW) {
      const T* src = static_cast<const T*>(a.h) + int64_t(m) * K + k0;
      for (int j = lane; j < KC; j += 32) hs[m * KC + j] = m < a.M && j < left ? Vec16<T>::load1(src + j) : 0.f;
    }
  };
  if (KC >= K) stage(0);
  __syncthreads();

  // This lane's values after the sum over lanes: (row r, token m) = lane * PER + i.
  XentRow xr[PER];
  int64_t target[PER];
  float run_m[PER], run_s[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int m = (lane * PER + i) % MT;
    run_m[i] = kNegInf, run_s[i] = 0.f;
    xr[i] = {0.f, 0.f, 0.f, -2};
    target[i] = -1;
    if (m < a.M) {
      if constexpr (GRAD) {
        xr[i] = a.row[m];
        target[i] = xr[i].target;
      } else {
        target[i] = a.targets[m];
      }
    }
  }

  const int64_t blocks = (a.V + R - 1) / R;
  for (int64_t b0 = int64_t(blockIdx.x) * NW; b0 < blocks; b0 += int64_t(gridDim.x) * NW) {  // the CTA's warps together
    const int64_t v0 = (b0 + warp) * R;
    const int rows = int(max(int64_t(0), min(int64_t(R), a.V - v0)));
    const T* w = static_cast<const T*>(a.w) + v0 * K;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    constexpr int kUnroll = KV == 4 ? 1 : 4;  // loads of w in flight: R kUnroll
    for (int64_t kc = 0; kc < K; kc += KC, w += KC) {  // k counts from kc: a sum of ints near 2^31 would not fit
      if (KC < K) {
        __syncthreads();
        stage(kc);
        __syncthreads();
      }
      const int end = int(min(int64_t(KC), K - kc));
      for (int k0 = lane * KV; k0 < end; k0 += 32 * KV * kUnroll) {
        float wv[kUnroll][R][KV];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int k = k0 + u * 32 * KV;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bool ok = k < end && r < rows;
            if constexpr (KV == 4) {
              const float4 x = ok ? __ldcs(reinterpret_cast<const float4*>(w + int64_t(r) * K + k)) : float4{};
              wv[u][r][0] = x.x, wv[u][r][1] = x.y, wv[u][r][2] = x.z, wv[u][r][3] = x.w;
            } else {
              wv[u][r][0] = ok ? Vec16<T>::load1(w + int64_t(r) * K + k) : 0.f;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int k = k0 + u * 32 * KV;
          if (k >= end) break;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float hv[KV];
            if constexpr (KV == 4) {
              const float4 x = *reinterpret_cast<const float4*>(hs + m * KC + k);
              hv[0] = x.x, hv[1] = x.y, hv[2] = x.z, hv[3] = x.w;
            } else {
              hv[0] = hs[m * KC + k];
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int c = 0; c < KV; ++c) acc[r * MT + m] = fmaf(wv[u][r][c], hv[c], acc[r * MT + m]);
          }
        }
      }
    }
    warp_transpose_sum<N>(acc, lane);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int idx = lane * PER + i, r = idx / MT, m = idx % MT;
      const int64_t v = v0 + r;
      if (r >= rows) continue;
      if constexpr (GRAD) {  // dloss (zf exp(x - lse) - onehot); zero for ignored rows and absent tokens
        float g = exp2_approx((acc[i] - xr[i].lse) * kLog2e) * xr[i].zf;
        if (v == target[i]) g -= 1.f;
        a.g[v0 * MT + idx] = xr[i].target == -2 ? 0.f : g * xr[i].g;
      } else if (m < a.M) {
        const float x = acc[i];
        if (v == target[i]) a.at_target[m] = x;
        const float mn = fmaxf(run_m[i], x);
        const float base = mn == kNegInf ? 0.f : mn * kLog2e;  // all -inf: a NaN still shows
        run_s[i] = (run_m[i] == kNegInf ? run_s[i] : run_s[i] * exp2_approx(fmaf(run_m[i], kLog2e, -base))) +
                   exp2_approx(fmaf(x, kLog2e, -base));
        run_m[i] = mn;
      }
    }
  }
  if constexpr (!GRAD) {
#pragma unroll
    for (int i = 0; i < PER; ++i) joint[warp][lane * PER + i] = make_float2(run_m[i], run_s[i]);
    __syncthreads();
    const int m = threadIdx.x;
    if (m >= a.M) return;
    float mx = kNegInf, s = 0.f;
    for (int k = 0; k < NW * R; ++k) mx = fmaxf(mx, joint[k / R][k % R * MT + m].x);
    for (int k = 0; k < NW * R; ++k) {  // in order
      const float2 p = joint[k / R][k % R * MT + m];
      s += p.x == kNegInf ? p.y : p.y * exp2_approx((p.x - mx) * kLog2e);
    }
    a.part[int64_t(blockIdx.x) * a.M + m] = make_float2(mx, s);
  }
}

// dh += g w and dw = g^T h in one walk over the vocabulary: a thread owns KV
// columns, whose h it keeps, and goes down the rows; g is read from shared memory
// by all threads at once.  A CTA of 256 threads takes `columns` threads across
// and 256 / columns rows at a time; each of those row lanes is a split of dh's sum.
template <typename T, int MT, int KV>
__global__ void __launch_bounds__(kFewThreads, 2) few_grad_kernel(const FewArgs a) {
  constexpr int kRows = 64;  // rows of g staged at a time
  __shared__ __align__(16) float gs[kRows][MT];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lanes = kFewThreads / a.columns, x = threadIdx.x % a.columns, y = threadIdx.x / a.columns;
  const int64_t k = (int64_t(blockIdx.x) * a.columns + x) * KV, K = a.K;
  const bool ok = k < K;  // K is a multiple of KV
  const int64_t begin = int64_t(blockIdx.y) * a.per_split, end = min(a.V, begin + a.per_split);
  const float f = *a.scale;
  float hv[MT][KV], acc[MT][KV];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < KV; ++c) {
      hv[m][c] = ok && m < a.M ? Vec16<T>::load1(static_cast<const T*>(a.h) + m * K + k + c) * f : 0.f;
      acc[m][c] = 0.f;
    }
  const T* w = static_cast<const T*>(a.w);
  T* dw = static_cast<T*>(a.dw);
  for (int64_t v0 = begin; v0 < end; v0 += kRows) {
    const int rows = int(min(int64_t(kRows), end - v0));
    __syncthreads();
    for (int e = threadIdx.x; e < rows * MT; e += kFewThreads) gs[e / MT][e % MT] = a.g[v0 * MT + e];
    __syncthreads();
    if (!ok) continue;
    constexpr int kUnroll = 8;
    for (int r0 = y; r0 < rows; r0 += lanes * kUnroll) {
      float wv[kUnroll][KV];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * lanes;
        const bool use = a.sum != nullptr && r < rows;
        const T* p = w + (v0 + r) * K + k;
        if constexpr (KV == 4) {
          const float4 q = use ? __ldcs(reinterpret_cast<const float4*>(p)) : float4{};
          wv[u][0] = q.x, wv[u][1] = q.y, wv[u][2] = q.z, wv[u][3] = q.w;
        } else if constexpr (KV == 2) {
          const float2 q = use ? __ldcs(reinterpret_cast<const float2*>(p)) : float2{};
          wv[u][0] = q.x, wv[u][1] = q.y;
        } else {
          wv[u][0] = use ? Vec16<T>::load1(p) : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int r = r0 + u * lanes;
        if (r >= rows) break;
        float d[KV] = {};
#pragma unroll
        for (int m = 0; m < MT; m += 4) {
          const float4 g4 = *reinterpret_cast<const float4*>(&gs[r][m]);
          const float g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < KV; ++c) {
              acc[m + e][c] = fmaf(g[e], wv[u][c], acc[m + e][c]);
              d[c] = fmaf(g[e], hv[m + e][c], d[c]);
            }
        }
        if (dw == nullptr) continue;
        T* p = dw + (v0 + r) * K + k;
        if constexpr (KV == 4) {
          __stcs(reinterpret_cast<float4*>(p), make_float4(d[0], d[1], d[2], d[3]));
        } else if constexpr (KV == 2) {
          __stcs(reinterpret_cast<float2*>(p), make_float2(d[0], d[1]));
        } else {
          Vec16<T>::store1(p, d[0]);
        }
      }
    }
  }
  if (a.sum == nullptr || !ok) return;
  float* s = a.sum + (int64_t(blockIdx.y) * lanes + y) * a.M * a.ld + k;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < KV; ++c)
      if (m < a.M) s[m * a.ld + c] = acc[m][c] * f;
}

}  // namespace qk
