// qk_quant.cu -- a matrix in 8 bits with a scale for each 128 elements of a row
// or each block of 128 x 128, straight and turned.
//
//   scale = max(max |x| of the group, 2^-100) / qmax,  q = rne(x / scale)
//
// Bound by memory: x is read once, q and its transpose are written once.  A CTA
// takes a tile of 128 x 128, which a group of any kind lies within: the tile
// stays in registers, so rows, columns and the block find their largest value in
// it and no element is loaded twice.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/qk.h"
#include "qk_host.h"
#include "qk_norm_kernels.cuh"  // scale_of, quotient, quantise2

namespace qk {
namespace {

constexpr int kTile = 128;
constexpr int kRows = 8;  // rows of a thread: with a 16-byte vector of each, 8 x 8 of bf16 or 8 x 4 of float32
template <typename T>
__host__ __device__ constexpr int quant_threads() { return kTile * kTile / kRows / (16 / int(sizeof(T))); }

struct QuantArgs {
  const void* x;   // [M, N]
  uint8_t* q;      // [M, N], may be null
  float* scale;
  uint8_t* qt;     // [N, M], may be null
  float* scale_t;
  int64_t M, N;
  int64_t col_tiles;
  int32_t block;   // nonzero: a scale a block of 128 x 128
  int32_t vec_q, vec_qt;  // rows of q (of qt) are whole 8-byte units
};

// The larger magnitude of two words of elements, a float or a bf16 pair, whatever
// its sign bits (magnitude() takes them off at the end); a NaN is larger than all.
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (sizeof(T) == 4) {
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  } else {
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  }
  return d;
}
// The largest magnitude among a word's elements, as a float.
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t w) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w & 0x7fffffffu);
  w &= 0x7fff7fffu;
  return __uint_as_float(max(w & 0xffff0000u, w << 16));
}

// What the values of one group are divided by: q = (x mul) / den with mul = qmax /
// 2^k (448 = 7 / 8 2^9, 127 = 127 / 128 2^7) and den = max |x| / 2^k, so that the
// quotient x qmax / max |x| is formed from exact numbers, not from a rounded scale,
// which would move one float32 value in a million to the other side of a tie.
struct Divisor {
  float den, inv;
};
template <int Q>
struct EightBitsOf {
  static constexpr float kMul = Q == QK_E4M3 ? 0.875f : 0.9921875f, kDown = Q == QK_E4M3 ? 0x1p-9f : 0x1p-7f;
  __device__ __forceinline__ static Divisor divisor(float amax, float* scale) {
    const bool bad = !(amax < __int_as_float(0x7f800000));
    *scale = scale_of(amax, bad, Q);
    const float den = bad ? *scale : fmaxf(amax, kSmallestGroupMax) * kDown;
    return {den, 1.f / den};
  }
  // The quotient x qmax / max |x| of a float32 x, rounded to float32: what is rounded to 8
  // bits.  What x mul's rounding left out joins the division's remainder; both are exact,
  // their sum and den's reciprocal to 2^-24.  So the rounded quotient is a or b, from
  // remainders 2^-20 apart on either side.  Where these are neighbours, what remains at the
  // point halfway between them decides, and is exact too: the quotient may be that point (3 as
  // a group's largest value has 33 such x beside ties of e4m3), and is the even one then.
  __device__ __forceinline__ static float value(float x, Divisor d) {
    const float y = x * kMul, q = quotient(y, d.den, d.inv);
    const float rem = fmaf(-q, d.den, y), low = fmaf(x, kMul, -y), s = rem + low;
    const float a = fmaf(s, d.inv * (1.f - 0x1p-20f), q), b = fmaf(s, d.inv * (1.f + 0x1p-20f), q);
    if (a == b) return a;
    const float left = fmaf(-((a - q) + 0.5f * (b - a)), d.den, rem) + low;
    return left > 0.f ? fmaxf(a, b) : left < 0.f ? fminf(a, b) : __float_as_uint(a) & 1u ? b : a;
  }
  // Four floats in 8 bits, the first in the low byte.
  __device__ __forceinline__ static uint32_t packed(const float* f) {
    if constexpr (Q == QK_INT8) return quantise2(f[0], f[1], Q) | quantise2(f[2], f[3], Q) << 16;
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]));
    return w;
  }
  // Four values of a group.  float32: from products with the rounded reciprocal, off by
  // less than 2^-22, where all that lies within 2^-21 of them rounds alike (all but
  // one value in 30000), else from the quotients (16384 x 4096 both ways with half
  // the threads: 139 us, from the quotients always 152).
  template <typename T>
  __device__ __forceinline__ static uint32_t four(const float* x, Divisor d) {
    float f[4];
    if constexpr (sizeof(T) == 4) {
      const float inv = kMul * d.inv;
      float g[4];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float2 q = mul2(make_float2(x[i], x[i + 1]), make_float2(inv, inv));
        const float2 lo = mul2(q, make_float2(1.f - 0x1p-21f, 1.f - 0x1p-21f)),
                     hi = mul2(q, make_float2(1.f + 0x1p-21f, 1.f + 0x1p-21f));
        f[i] = lo.x, f[i + 1] = lo.y, g[i] = hi.x, g[i + 1] = hi.y;
      }
      const uint32_t w = packed(f);
      if (w == packed(g)) return w;
    }
    if constexpr (sizeof(T) == 2) {
      // quotient() in packed pairs, as what bounds the kernel is the number of instructions.
      // x mul is exact, and no quotient of two float32 numbers is a halfway point.
      const float2 mul = make_float2(kMul, kMul), inv = make_float2(d.inv, d.inv), less = make_float2(-d.den, -d.den);
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float2 y = mul2(make_float2(x[i], x[i + 1]), mul), q = mul2(y, inv), r = fma2(fma2(q, less, y), inv, q);
        f[i] = r.x, f[i + 1] = r.y;
      }
    } else {
      // Small groups are taken 2^64 times as large, so that no remainder underflows.
      const bool small = d.den < 0x1p-60f;
      const float up = small ? 0x1p64f : 1.f;
      const Divisor e = {d.den * up, small ? d.inv * 0x1p-64f : d.inv};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = value(x[i] * up, e);
    }
    return packed(f);
  }
};

// E (8 or 4) values in 8 bits.
template <int E>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t* words) {
  if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(words[0], words[1]);
  else *reinterpret_cast<uint32_t*>(p) = words[0];
}

// A row of n <= 128 bytes that starts anywhere, by a warp: words where the memory has
// them, bytes at the ends.  word(i) is the row's i-th word in shared memory
// (16384 x 4095 bf16, straight: 95 us, 128 with bytes; 16383 x 4096 turned: 62 and 100).
template <typename F>
__device__ __forceinline__ void store_row(uint8_t* p, int n, int lane, F word) {
  const int lead = min(n, int(-reinterpret_cast<uintptr_t>(p) & 3)), words = (n - lead) >> 2, tail = lead + 4 * words;
  auto byte = [&](int i) { return uint8_t(word(i >> 2) >> (8 * (i & 3))); };
  if (lane < words)
    *reinterpret_cast<uint32_t*>(p + lead + 4 * lane) =
        __funnelshift_r(word(lane), lead == 0 || lane == 31 ? 0u : word(lane + 1), 8 * lead);
  if (lane < lead) p[lane] = byte(lane);
  if (tail + lane < n) p[tail + lane] = byte(tail + lane);
}

// 16 bytes from anywhere in [lo, hi), from the words that they lie in, which the matrix
// has to hold; false where it does not.
__device__ __forceinline__ bool load_across(const void* p, uintptr_t lo, uintptr_t hi, uint4* v) {
  const uintptr_t s = reinterpret_cast<uintptr_t>(p), s4 = s & ~uintptr_t(3);
  const uint32_t shift = uint32_t(s & 3) * 8;
  if (s4 < lo || s4 + (shift == 0 ? 16 : 20) > hi) return false;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(s4);
  const uint32_t a = w[0], b = w[1], c = w[2], d = w[3], e = shift == 0 ? 0 : w[4];
  *v = make_uint4(__funnelshift_r(a, b, shift), __funnelshift_r(b, c, shift), __funnelshift_r(c, d, shift),
                  __funnelshift_r(d, e, shift));
  return true;
}

// The registers of a thread are held down to 64 (bf16: 62 us at 16384 x 4096 both
// ways, 66 with 85 and three CTAs an SM).
template <typename T, int Q, bool VEC>
__global__ void __launch_bounds__(quant_threads<T>(), 1024 / quant_threads<T>()) quant_kernel(const QuantArgs a) {
  using V = Vec16<T>;
  using B = EightBitsOf<Q>;
  constexpr int E = V::kElems, kLanes = kTile / E, R = kRows, kWarps = quant_threads<T>() / 32;
  constexpr int kShare = kLanes / R;  // lanes that end with one row's largest
  __shared__ __align__(16) uint4 tops[kWarps][kLanes];   // largest bits of a warp's rows, by column
  __shared__ uint32_t warp_top[kWarps];
  __shared__ Divisor columns[kTile];
  __shared__ __align__(16) uint8_t turned[kTile * kTile];
  grid_dependency_wait();
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t mt = int64_t(blockIdx.x) / a.col_tiles, nt = int64_t(blockIdx.x) - mt * a.col_tiles;
  const int64_t i0 = mt * kTile, j0 = nt * kTile, row_tiles = (a.M + kTile - 1) / kTile;
  const int r0 = (warp * (32 / kLanes) + lane / kLanes) * R, c0 = (lane % kLanes) * E;  // this thread's part of the tile
  const int rows = int(min(int64_t(kTile), a.M - i0)), cols = int(min(int64_t(kTile), a.N - j0));
  const T* x = static_cast<const T*>(a.x) + (i0 + r0) * a.N + j0 + c0;

  uint4 raw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    raw[r] = make_uint4(0, 0, 0, 0);
    if (r0 + r < rows) {
      if constexpr (VEC) {  // N is a multiple of E
        if (c0 < cols) raw[r] = __ldcs(reinterpret_cast<const uint4*>(x + r * a.N));
      } else {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(a.x), hi = lo + uintptr_t(a.M) * uintptr_t(a.N) * sizeof(T);
        if (sizeof(T) == 4 || c0 + E > cols || !load_across(x + r * a.N, lo, hi, &raw[r])) {
          float f[E];
#pragma unroll
          for (int j = 0; j < E; ++j) f[j] = c0 + j < cols ? V::load1(x + r * a.N + j) : 0.f;
          raw[r] = V::pack(f);  // exact: the values are T's
        }
      }
    }
  }

  uint32_t row_top[R];
  uint4 col_top = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint4 m = raw[r];
    row_top[r] = larger<T>(larger<T>(m.x, m.y), larger<T>(m.z, m.w));
    col_top = make_uint4(larger<T>(col_top.x, m.x), larger<T>(col_top.y, m.y), larger<T>(col_top.z, m.z),
                         larger<T>(col_top.w, m.w));
  }
  if (a.qt != nullptr && !a.block) {
    if constexpr (kLanes == 16) {
      col_top.x = larger<T>(col_top.x, __shfl_xor_sync(0xffffffffu, col_top.x, 16));
      col_top.y = larger<T>(col_top.y, __shfl_xor_sync(0xffffffffu, col_top.y, 16));
      col_top.z = larger<T>(col_top.z, __shfl_xor_sync(0xffffffffu, col_top.z, 16));
      col_top.w = larger<T>(col_top.w, __shfl_xor_sync(0xffffffffu, col_top.w, 16));
    }
    if (lane < kLanes) tops[warp][lane] = col_top;
  }
  // The rows' largest over their kLanes lanes: each step hands half of the rows to
  // the other lane, so that kShare lanes end with one row, in some R shuffles
  // instead of R log2(kLanes).
#pragma unroll
  for (int n = R / 2, o = kLanes / 2; n >= 1; n /= 2, o /= 2) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const uint32_t send = upper ? row_top[i] : row_top[i + n], keep = upper ? row_top[i + n] : row_top[i];
      row_top[i] = larger<T>(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
#pragma unroll
  for (int o = kShare / 2; o >= 1; o /= 2) row_top[0] = larger<T>(row_top[0], __shfl_xor_sync(0xffffffffu, row_top[0], o));
  const float own = magnitude<T>(row_top[0]);  // of row (lane % kLanes) / kShare of this group of lanes
  float scale;
  Divisor block = {1.f, 1.f};
  if (a.block) {
    uint32_t top = __float_as_uint(own);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) warp_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, warp_top[w]);
    block = B::divisor(__uint_as_float(top), &scale);
    if (threadIdx.x == 0) {
      if (a.q != nullptr) a.scale[mt * a.col_tiles + nt] = scale;
      if (a.qt != nullptr) a.scale_t[nt * row_tiles + mt] = scale;
    }
  }
  if (a.q != nullptr) {
    Divisor mine = block;
    if (!a.block) {
      mine = B::divisor(own, &scale);
      const int row = r0 + (lane % kLanes) / kShare;
      if (lane % kShare == 0 && row < rows) a.scale[(i0 + row) * a.col_tiles + nt] = scale;
    }
    uint8_t* q = a.q + (i0 + r0) * a.N + j0 + c0;
    const bool inside = a.vec_q && rows == kTile && cols == kTile;
#pragma unroll
    for (int r = 0; r < R; ++r, q += a.N) {
      const int from = (lane & ~(kLanes - 1)) + kShare * r;
      const Divisor d = {__shfl_sync(0xffffffffu, mine.den, from), __shfl_sync(0xffffffffu, mine.inv, from)};
      float f[E];
      V::unpack(raw[r], f);
      uint32_t words[E / 4];
#pragma unroll
      for (int j = 0; j < E; j += 4) words[j / 4] = B::template four<T>(f + j, d);
      if (inside || (a.vec_q && r0 + r < rows && c0 < cols)) {
        store_words<E>(q, words);  // N is a multiple of 8
      } else if (!a.vec_q && sizeof(T) == 2) {
        store_words<E>(turned + (r0 + r) * kTile + c0, words);
      } else if (!a.vec_q && r0 + r < rows) {  // float32's four bytes a thread: 79 us at 16384 x 4095, by way of the tile 99
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (c0 + j < cols) q[j] = uint8_t(words[j / 4] >> (8 * (j % 4)));
      }
    }
    if (!a.vec_q && sizeof(T) == 2) {
      __syncthreads();
      for (int row = warp; row < rows; row += kWarps)
        store_row(a.q + (i0 + row) * a.N + j0, cols, lane,
                  [&](int i) { return reinterpret_cast<const uint32_t*>(turned + row * kTile)[i]; });
      __syncthreads();
    }
  }
  if (a.qt == nullptr) return;
  if (!a.block) {
    __syncthreads();
    if (threadIdx.x < kTile) {
      const int c = threadIdx.x;
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if constexpr (sizeof(T) == 4) top = max(top, reinterpret_cast<const uint32_t*>(tops[w])[c] & 0x7fffffffu);
        else top = max(top, (uint32_t(reinterpret_cast<const uint16_t*>(tops[w])[c]) & 0x7fffu) << 16);
      }
      columns[c] = B::divisor(__uint_as_float(top), &scale);
      if (c < cols) a.scale_t[(j0 + c) * row_tiles + mt] = scale;
    }
    __syncthreads();
  }
  // Columns as rows of bytes.  Units of 8 rows are XORed with the columns' number
  // / 8: lanes of one store hit different banks, and so do those of one load.
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const Divisor d = a.block ? block : columns[c0 + j];
    const int unit_key = (c0 + j) >> 3;
    uint32_t words[2];
#pragma unroll
    for (int r = 0; r < R; r += 4) {
      float column[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[E];
        V::unpack(raw[r + i], f);
        column[i] = f[j];
      }
      words[r / 4] = B::template four<T>(column, d);
    }
    *reinterpret_cast<uint2*>(turned + (c0 + j) * kTile + (((r0 >> 3) ^ unit_key) & 15) * 8) = make_uint2(words[0], words[1]);
  }
  __syncthreads();
  if (!a.vec_qt) {
    for (int col = warp; col < cols; col += kWarps)
      store_row(a.qt + (j0 + col) * a.M + i0, rows, lane, [&](int i) {
        return *reinterpret_cast<const uint32_t*>(turned + col * kTile + (((i >> 1) ^ (col >> 3)) & 15) * 8 + (i & 1) * 4);
      });
    return;
  }
  const int unit = lane & 15, first = warp * 2 + (lane >> 4);
  uint8_t* qt = a.qt + (j0 + first) * a.M + i0 + unit * 8;
  const bool inside = rows == kTile && cols == kTile;
#pragma unroll
  for (int k = 0; k < kTile / 2 / kWarps; ++k, qt += 2 * kWarps * a.M) {
    const int col = first + k * 2 * kWarps;
    const uint2 w = *reinterpret_cast<const uint2*>(turned + col * kTile + ((unit ^ (col >> 3)) & 15) * 8);
    const uint32_t words[2] = {w.x, w.y};
    if (inside || (col < cols && unit * 8 < rows)) store_words<8>(qt, words);  // M is a multiple of 8
  }
}

template <typename T, int Q>
qk_status launch_quant(const QuantArgs& a, bool vec, int64_t tiles, void* stream) {
  const auto kernel = vec ? quant_kernel<T, Q, true> : quant_kernel<T, Q, false>;
  return launch_pdl(kernel, dim3(unsigned(tiles)), quant_threads<T>(), 0, stream, a);
}
template <typename T>
qk_status launch_quant(const QuantArgs& a, int qtype, bool vec, int64_t tiles, void* stream) {
  return qtype == QK_E4M3 ? launch_quant<T, QK_E4M3>(a, vec, tiles, stream)
                          : launch_quant<T, QK_INT8>(a, vec, tiles, stream);
}

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" qk_status qk_quant_fwd(const void* x, void* q, float* scale, void* qt, float* scale_t, int64_t M, int64_t N,
                                  int64_t block_rows, qk_dtype dtype, qk_qtype qtype, void* stream) {
  if (dtype != QK_F32 && dtype != QK_BF16) return QK_ERR_INVALID_ARG;
  if (qtype != QK_E4M3 && qtype != QK_INT8) return QK_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != 128) return QK_ERR_INVALID_ARG;
  if (M < 0 || N <= 0 || M > INT64_MAX / 16 / N) return QK_ERR_INVALID_ARG;
  if ((q == nullptr) != (scale == nullptr) || (qt == nullptr) != (scale_t == nullptr)) return QK_ERR_INVALID_ARG;
  if (M == 0) return QK_OK;
  if (x == nullptr || (q == nullptr && qt == nullptr)) return QK_ERR_INVALID_ARG;
  const size_t es = size_t(elem_size(dtype));
  if (!aligned_to(x, es) || !aligned_to(scale, 4) || !aligned_to(scale_t, 4)) return QK_ERR_MISALIGNED;
  const int64_t row_tiles = (M + kTile - 1) / kTile, col_tiles = (N + kTile - 1) / kTile;
  if (row_tiles > INT32_MAX / col_tiles) return QK_ERR_UNSUPPORTED;
  const int64_t sb = (block_rows == 1 ? M : row_tiles) * col_tiles * 4, tb = (block_rows == 1 ? N : col_tiles) * row_tiles * 4;
  const struct {
    const void* p;
    int64_t n;
  } out[] = {{q, M * N}, {scale, sb}, {qt, M * N}, {scale_t, tb}};
  for (int i = 0; i < 4; ++i) {
    if (overlap(out[i].p, out[i].n, x, M * N * int64_t(es))) return QK_ERR_INVALID_ARG;
    for (int k = i + 1; k < 4; ++k)
      if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return QK_ERR_INVALID_ARG;
  }
  CurrentDevice d;
  const qk_status st = current_device(&d);
  if (st != QK_OK) return st;
  QuantArgs a = {};
  a.x = x;
  a.q = static_cast<uint8_t*>(q);
  a.scale = scale;
  a.qt = static_cast<uint8_t*>(qt);
  a.scale_t = scale_t;
  a.M = M;
  a.N = N;
  a.col_tiles = col_tiles;
  a.block = block_rows == 128;
  a.vec_q = N % 8 == 0 && aligned_to(q, 8);
  a.vec_qt = M % 8 == 0 && aligned_to(qt, 8);
  const bool vec = N * int64_t(es) % 16 == 0 && aligned16(x);
  return dtype == QK_F32 ? launch_quant<float>(a, qtype, vec, row_tiles * col_tiles, stream)
                         : launch_quant<__nv_bfloat16>(a, qtype, vec, row_tiles * col_tiles, stream);
}
