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
#include "qk_norm_kernels.cuh"  // EightBits, quotient, quantise2

namespace qk {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kTile = 128;

struct QuantArgs {
  const void* x;   // [M, N]
  uint8_t* q;      // [M, N], may be null
  float* scale;
  uint8_t* qt;     // [N, M], may be null
  float* scale_t;
  int64_t M, N;
  int64_t col_tiles;
  int32_t block;   // nonzero: a scale a block of 128 x 128
  int32_t qtype;
  int32_t vec_q, vec_qt;  // rows of q (of qt) are whole 8-byte units
};

// Bits of |x|, which compare as |x| does, with a NaN above all numbers.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <int WIDTH>
__device__ __forceinline__ uint32_t group_max_bits(uint32_t v) {
#pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// One row of `n` (8 or 4) values in 8 bits, from the values as floats.
template <int E>
__device__ __forceinline__ void store_bytes(uint8_t* p, const uint32_t* words, int left, bool vec) {
  if (vec && left >= E) {
    if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(words[0], words[1]);
    else *reinterpret_cast<uint32_t*>(p) = words[0];
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (j < left) p[j] = uint8_t(words[j / 4] >> (8 * (j % 4)));
}

// A thread holds E columns (a 16-byte vector) of R rows that follow each other:
// 8 x 8 of bf16, 16 x 4 of float32.  A warp has 16 rows of the tile.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads, 2) quant_kernel(const QuantArgs a) {
  using V = Vec16<T>;
  constexpr int E = V::kElems, kLanes = kTile / E, R = 16 * kLanes / 32;
  __shared__ uint32_t tops[8][kTile];     // largest bits of a warp's rows, by column
  __shared__ __align__(16) uint8_t turned[kTile * kTile];
  grid_dependency_wait();
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t mt = int64_t(blockIdx.x) / a.col_tiles, nt = int64_t(blockIdx.x) - mt * a.col_tiles;
  const int64_t i0 = mt * kTile, j0 = nt * kTile;
  const int r0 = warp * 16 + (lane / kLanes) * R, c0 = (lane % kLanes) * E;  // this thread's part of the tile
  const int rows = int(min(int64_t(kTile), a.M - i0)), cols = int(min(int64_t(kTile), a.N - j0));
  const T* x = static_cast<const T*>(a.x) + (i0 + r0) * a.N + j0 + c0;

  uint4 raw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    raw[r] = make_uint4(0, 0, 0, 0);
    if (r0 + r < rows) {
      if constexpr (VEC) {  // N is a multiple of E
        if (c0 < cols) raw[r] = *reinterpret_cast<const uint4*>(x + r * a.N);
      } else {
        float f[E];
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = c0 + j < cols ? V::load1(x + r * a.N + j) : 0.f;
        raw[r] = V::pack(f);  // exact: the values are T's
      }
    }
  }
  const EightBits<T> bits(1.f, a.qtype);
  const int groups = int(a.col_tiles);

  uint32_t row_top[R], col_top[E];
#pragma unroll
  for (int j = 0; j < E; ++j) col_top[j] = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float f[E];
    V::unpack(raw[r], f);
    row_top[r] = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const uint32_t m = magnitude(f[j]);
      row_top[r] = max(row_top[r], m);
      col_top[j] = max(col_top[j], m);
    }
  }
  uint32_t block_top = 0;
  if (a.block || a.qt != nullptr) {
    if constexpr (kLanes == 16) {
#pragma unroll
      for (int j = 0; j < E; ++j) col_top[j] = max(col_top[j], __shfl_xor_sync(0xffffffffu, col_top[j], 16));
    }
    if (lane < kLanes) {
#pragma unroll
      for (int j = 0; j < E; ++j) tops[warp][c0 + j] = col_top[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) {
#pragma unroll
      for (int w = 0; w < 8; ++w) col_top[j] = max(col_top[j], tops[w][c0 + j]);
      block_top = max(block_top, col_top[j]);
    }
    block_top = group_max_bits<kLanes>(block_top);
  }

  // The largest |x mul|, as EightBits wants it, and what a value is divided by.
  auto denominator = [&](uint32_t top, float* scale) {
    float den;
    *scale = bits.scale(__uint_as_float(top) * bits.mul, a.qtype, &den);
    return den;
  };
  float scale, den_block = 0.f;
  if (a.block) {
    den_block = denominator(block_top, &scale);
    if (threadIdx.x == 0) {
      const int64_t row_tiles = (a.M + kTile - 1) / kTile;
      if (a.q != nullptr) a.scale[mt * groups + nt] = scale;
      if (a.qt != nullptr) a.scale_t[nt * row_tiles + mt] = scale;
    }
  }
  if (a.q != nullptr) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float den = den_block;
      if (!a.block) {
        den = denominator(group_max_bits<kLanes>(row_top[r]), &scale);
        if (lane % kLanes == 0 && r0 + r < rows) a.scale[(i0 + r0 + r) * groups + nt] = scale;
      }
      const float inv = EightBits<T>::inverse(den);
      float f[E];
      V::unpack(raw[r], f);
      uint32_t words[E / 4];
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        words[j / 4] = quantise2(quotient(f[j] * bits.mul, den, inv), quotient(f[j + 1] * bits.mul, den, inv), a.qtype) |
                       quantise2(quotient(f[j + 2] * bits.mul, den, inv), quotient(f[j + 3] * bits.mul, den, inv), a.qtype) << 16;
      }
      if (r0 + r < rows) store_bytes<E>(a.q + (i0 + r0 + r) * a.N + j0 + c0, words, cols - c0, a.vec_q);
    }
  }
  if (a.qt != nullptr) {
    const int64_t row_tiles = (a.M + kTile - 1) / kTile;
    // Columns as rows of bytes.  Units of 8 rows are XORed with the columns' number
    // / 8: lanes of one store hit different banks, and so do those of one load.
#pragma unroll
    for (int j = 0; j < E; ++j) {
      float den = den_block;
      if (!a.block) {
        den = denominator(col_top[j], &scale);
        if (r0 == 0 && c0 + j < cols) a.scale_t[(j0 + c0 + j) * row_tiles + mt] = scale;
      }
      const float inv = EightBits<T>::inverse(den);
      const int unit_key = (c0 + j) >> 3;
#pragma unroll
      for (int u = 0; u < R / 8; ++u) {
        uint32_t words[2] = {0, 0};
#pragma unroll
        for (int r = 0; r < 8; r += 2) {
          float f[E], g[E];
          V::unpack(raw[u * 8 + r], f);
          V::unpack(raw[u * 8 + r + 1], g);
          words[r / 4] |= quantise2(quotient(f[j] * bits.mul, den, inv), quotient(g[j] * bits.mul, den, inv), a.qtype)
                          << (8 * (r % 4));
        }
        const int unit = (r0 >> 3) + u;
        *reinterpret_cast<uint2*>(turned + (c0 + j) * kTile + ((unit ^ unit_key) & 15) * 8) = make_uint2(words[0], words[1]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int col = k * 16 + warp * 2 + (lane >> 4), unit = lane & 15;
      const uint2 w = *reinterpret_cast<const uint2*>(turned + col * kTile + ((unit ^ (col >> 3)) & 15) * 8);
      const uint32_t words[2] = {w.x, w.y};
      if (col < cols && unit * 8 < rows)
        store_bytes<8>(a.qt + (j0 + col) * a.M + i0 + unit * 8, words, rows - unit * 8, a.vec_qt);
    }
  }
}

template <typename T>
qk_status launch_quant(const QuantArgs& a, bool vec, int64_t tiles, void* stream) {
  const auto kernel = vec ? quant_kernel<T, true> : quant_kernel<T, false>;
  return launch_pdl(kernel, dim3(unsigned(tiles)), kQuantThreads, 0, stream, a);
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
  a.qtype = qtype;
  a.vec_q = N % 8 == 0 && aligned_to(q, 8);
  a.vec_qt = M % 8 == 0 && aligned_to(qt, 8);
  const bool vec = N * int64_t(es) % 16 == 0 && aligned16(x);
  return dtype == QK_F32 ? launch_quant<float>(a, vec, row_tiles * col_tiles, stream)
                         : launch_quant<__nv_bfloat16>(a, vec, row_tiles * col_tiles, stream);
}
