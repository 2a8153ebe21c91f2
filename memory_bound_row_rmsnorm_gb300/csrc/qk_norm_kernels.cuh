// qk_norm_kernels.cuh -- RMSNorm with the residual's addition: forward, forward
// with an 8-bit output, and backward (sm_103a).
//
//   h = rnd(x + r),  rstd = (mean h^2 + eps)^-1/2,  y = h rstd w
//   q = rne(y / scale), scale = max(max |y|, 2^-100) / qmax per row or group of columns
//   dx = dh + rstd dy w - h rstd^3 mean(dy w h),  dw = sum over rows of dy h rstd
//
// All three are bound by memory: a handful of operations for the 2 to 4
// matrices that pass through.
#pragma once

#include <cuda_fp8.h>

#include "qk_device.cuh"
#include "qk_internal.h"

namespace qk {

enum NormOp : int { kAddNorm = 0, kNormQuant = 1, kAddNormBwd = 2 };

constexpr float kSmallestGroupMax = 0x1p-100f;  // no group's largest |y| counts as less

struct NormArgs {
  const void* x;     // [M, N] x (forward) or h (backward)
  const void* r;     // [M, N] residual (forward, may be null) or dy (backward)
  const void* r2;    // [M, N] dh (backward, may be null)
  const void* w;     // [N]
  void* y;           // [M, N] y, q or dx
  void* h;           // [M, N] forward: the kept sum, may be null
  float* scale;      // [M, groups] 8-bit output
  float* rstd;       // [M] written by the forward (may be null), read by the backward
  float* dw_partial; // [partial rows, N] backward
  int64_t M, N;
  int64_t groups;    // scales of one row
  int32_t group;     // columns of one scale, 0: the row
  int32_t qtype;     // QK_E4M3 or QK_INT8
  float eps;
  float inv_n;       // 1 / N
  int32_t slots;        // ring slots (ring kernel)
  uint32_t slot_bytes;  // bytes of one input's item in a slot
  int64_t num_items;
  uint64_t timeout_ns;
  int* status;
};

__device__ __forceinline__ float qmax_of(int qtype) { return qtype == 0 ? 448.f : 127.f; }
// y / s with inv = 1 / s rounded: the product's residual corrects it (Markstein's
// division step), so that what is rounded to 8 bits is the rounded quotient, not
// one that the reciprocal's rounding moved across a tie.  A NaN s stays NaN.
__device__ __forceinline__ float quotient(float y, float s, float inv) {
  const float q = y * inv;
  return fmaf(fmaf(-q, s, y), inv, q);
}
// The scale of a group from its largest |y|; `bad` when a y of the group is not
// finite.  By quotient(), which is the rounded division for all of these (every
// significand was tried), in a third of a division's instructions.
__device__ __forceinline__ float scale_of(float amax, bool bad, int qtype) {
  const float s = quotient(fmaxf(amax, kSmallestGroupMax), qmax_of(qtype), qtype == 0 ? 1.f / 448.f : 1.f / 127.f);
  return bad ? __int_as_float(0x7fc00000) : s;
}

// An element of a row on its way to 8 bits, and the scale of a group of them.
// Each stands as (h mul) w, of which scale() gets the group's largest; what is
// rounded is quotient((h mul) w, den, 1 / den).
//
// float32: that is y, and den is the scale.
// bf16: a product h w has 16 bits of significand, and of y = h rstd w only rstd
// has more, which the quotient does not depend on.  So rstd is left out but for
// its power of two: mul = 2^e qmax / 2^k (448 = 7 / 8 2^9, 127 = 127 / 128 2^7)
// makes y' = (h mul) w exact in 23 bits, and y / scale = y' / (max |h 2^e w| / 2^k)
// is one division of exact numbers.  A quotient that lies on a tie is one
// then, and goes to even.  From a rounded y it goes to either side with the last
// bit of rstd, which the order of a row's sum decides: at 16384 x 4096 one
// value in 10000 lies on a tie, and their error was 8.7e-4 of q's norm.
template <typename T>
struct EightBits {
  float mul, rest = 1.f, low = 0.f;  // y = (h mul) w 2^k / qmax * rest; low: kSmallestGroupMax / rest
  __device__ __forceinline__ EightBits(float rs, int qtype) : mul(rs) {
    if constexpr (sizeof(T) == 2) {  // rs is 0, infinite, NaN or a normal number: 1 / sqrt of a float32
      const uint32_t b = __float_as_uint(rs);
      mul = __uint_as_float(b & 0x7f800000u) * (qtype == 0 ? 0.875f : 0.9921875f);
      rest = __uint_as_float((b & 0x007fffffu) | 0x3f800000u);
      low = kSmallestGroupMax / rest;
    }
  }
  __device__ __forceinline__ float scale(float m, int qtype, float* den) const {
    if constexpr (sizeof(T) == 4) {
      return *den = scale_of(m, !(m < __int_as_float(0x7f800000)), qtype);
    } else {
      // m 2^k / qmax = m + m / 7 or m + m / 127, a number of 16 bits: the
      // constant's rounding is 2^-27 or less of the sum and does not show.
      const float top = fmaf(m, qtype == 0 ? 1.f / 7.f : 1.f / 127.f, m);
      const float amax = top * rest;
      const bool bad = !(amax < __int_as_float(0x7f800000));
      const float s = scale_of(amax, bad, qtype);
      *den = bad ? s : fmaxf(top, low) * (qtype == 0 ? 0x1p-9f : 0x1p-7f);
      return s;
    }
  }
  // 1 / den.  For bf16 den is below 2^122, far from where the approximation
  // ends, and a step of Newton's is enough: quotient() finds a tie from any
  // reciprocal within a bit or two.
  __device__ __forceinline__ static float inverse(float den) {
    if constexpr (sizeof(T) == 4) return 1.f / den;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(den));
    return fmaf(fmaf(-den, r, 1.f), r, r);
  }
};
// One value in 8 bits, to nearest even.  |v| exceeds qmax by rounding at most, which saturates.
__device__ __forceinline__ uint32_t quantise(float v, int qtype) {
  if (qtype == 0) return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
  return uint32_t(max(-127, min(127, __float2int_rn(v)))) & 0xffu;  // NaN converts to 0
}

// Two of them, the first in the low byte.
__device__ __forceinline__ uint32_t quantise2(float a, float b, int qtype) {
  if (qtype == 0) return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  return quantise(a, 1) | quantise(b, 1) << 8;
}

// x + r rounded to the rows' type, as a float.
template <typename T>
__device__ __forceinline__ float rounded_sum(float x, float r) {
  if constexpr (sizeof(T) == 4) return x + r;
  return __bfloat162float(__float2bfloat16_rn(x + r));
}

// Sum (or maximum) over the CTA, the same bits in every thread; `red` holds
// THREADS / 32 floats and may be used again after the next __syncthreads.
template <int THREADS>
__device__ __forceinline__ float cta_sum(float v, float* red) {
  v = group_sum<32>(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) s += red[i];
  return s;
}
template <int THREADS>
__device__ __forceinline__ float cta_max(float v, float* red) {
  v = group_max<32>(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) s = fmaxf(s, red[i]);
  return s;
}

// ---------------------------------------------------------------------------
// Any row: one CTA walks rows with element loads, two or three passes a row.
// The second pass reads the kept h, or x and r again, which are in L1 or L2
// by then.  Nothing here depends on alignment or on the row's length.
// ---------------------------------------------------------------------------
constexpr int kNormAnyThreads = 256;

template <int OP, typename T>
__global__ void __launch_bounds__(kNormAnyThreads) norm_any_kernel(const NormArgs a) {
  using V = Vec16<T>;
  constexpr int TH = kNormAnyThreads;
  __shared__ float red[3][TH / 32];
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t N = a.N;
  const T* w = static_cast<const T*>(a.w);
  float* part = OP == kAddNormBwd ? a.dw_partial + int64_t(blockIdx.x) * N : nullptr;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    // no __restrict__: h may be x or r, y may be x or r, dx may be any input
    const T* x = static_cast<const T*>(a.x) + row * N;
    const T* r = a.r != nullptr ? static_cast<const T*>(a.r) + row * N : nullptr;
    T* h = OP != kAddNormBwd && a.h != nullptr ? static_cast<T*>(a.h) + row * N : nullptr;
    __syncthreads();  // the last row's use of `red`, and its h
    if constexpr (OP == kAddNormBwd) {
      const T* dh = a.r2 != nullptr ? static_cast<const T*>(a.r2) + row * N : nullptr;
      T* dx = static_cast<T*>(a.y) + row * N;
      const float rs = a.rstd[row];
      float dot = 0.f;
      for (int64_t j = tid; j < N; j += TH) dot = fmaf(V::load1(r + j) * V::load1(w + j), V::load1(x + j), dot);
      const float c = (cta_sum<TH>(dot, red[0]) * a.inv_n) * rs * rs * rs;  // in this order, as in the ring kernel
      const bool first = row == blockIdx.x;
      for (int64_t j = tid; j < N; j += TH) {
        const float hv = V::load1(x + j), dy = V::load1(r + j);
        const float up = dh != nullptr ? V::load1(dh + j) : 0.f;
        V::store1(dx + j, up + fmaf(hv, -c, (rs * dy) * V::load1(w + j)));
        const float p = (dy * hv) * rs;  // this thread's columns are its own in every row
        part[j] = first ? p : part[j] + p;
      }
    } else {
      auto value = [&](int64_t j) {  // the kept h at column j
        const float xv = V::load1(x + j);
        return r != nullptr ? rounded_sum<T>(xv, V::load1(r + j)) : xv;
      };
      float ss = 0.f;
      for (int64_t j = tid; j < N; j += TH) {
        const float v = value(j);
        if (h != nullptr) V::store1(h + j, v);
        ss = fmaf(v, v, ss);
      }
      const float rs = 1.f / sqrtf(fmaf(cta_sum<TH>(ss, red[0]), a.inv_n, a.eps));
      if (tid == 0 && a.rstd != nullptr) a.rstd[row] = rs;
      // From here on h (when kept) is what is read: x or r may be gone.
      auto scaled = [&](int64_t j, float f) { return (h != nullptr ? V::load1(h + j) : value(j)) * f * V::load1(w + j); };
      if constexpr (OP == kAddNorm) {
        T* y = static_cast<T*>(a.y) + row * N;
        for (int64_t j = tid; j < N; j += TH) V::store1(y + j, scaled(j, rs));
      } else {
        uint8_t* q = static_cast<uint8_t*>(a.y) + row * N;
        float* sc = a.scale + row * a.groups;
        const EightBits<T> eight(rs, a.qtype);
        constexpr float kNan = __builtin_nanf("");
        if (a.group == 0) {
          float m = 0.f, bad = 0.f;
          for (int64_t j = tid; j < N; j += TH) {
            const float v = fabsf(scaled(j, eight.mul));
            m = fmaxf(m, v);
            if (!(v < __int_as_float(0x7f800000))) bad = 1.f;
          }
          m = cta_max<TH>(m, red[1]);
          bad = cta_max<TH>(bad, red[2]);
          float den;
          const float s = eight.scale(bad > 0.f ? kNan : m, a.qtype, &den);
          if (tid == 0) sc[0] = s;
          const float inv = eight.inverse(den);
          for (int64_t j = tid; j < N; j += TH)
            q[j] = uint8_t(quantise(quotient(scaled(j, eight.mul), den, inv), a.qtype));
        } else {
          __syncthreads();  // a warp reads what others kept of h
          for (int64_t g = warp; g < a.groups; g += TH / 32) {
            float v[4], m = 0.f;
            bool bad = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // a group has at most 128 columns
              const int64_t j = g * a.group + lane + 32 * k;
              v[k] = 32 * k < a.group && j < N ? scaled(j, eight.mul) : 0.f;
              m = fmaxf(m, fabsf(v[k]));
              bad |= !(fabsf(v[k]) < __int_as_float(0x7f800000));
            }
            m = group_max<32>(m);
            float den;
            const float s = eight.scale(__any_sync(0xffffffffu, bad) ? kNan : m, a.qtype, &den);
            if (lane == 0) sc[g] = s;
            const float inv = eight.inverse(den);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int64_t j = g * a.group + lane + 32 * k;
              if (32 * k < a.group && j < N) q[j] = uint8_t(quantise(quotient(v[k], den, inv), a.qtype));
            }
          }
        }
      }
    }
  }
}

}  // namespace qk
