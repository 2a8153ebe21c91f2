// qk_norm_ring.cuh -- the ring kernel of the norms with the residual's
// addition: rows held in registers, one pass over memory (sm_103a).
//
// A persistent grid; in each CTA one thread streams work items (a block of
// THREADS / TPR rows of every input) into a shared-memory ring with
// cp.async.bulk under mbarriers, TPR threads share a row, and every output is
// stored once.  What bounds it is HBM: 2 to 4 matrices in and out, some ten
// operations an element.
//
// VEC: rows of whole 16-byte vectors; a thread works on vectors l + k TPR.
// Otherwise a thread works on elements l + k TPR of rows that start anywhere: an
// item is copied as the 16-byte aligned range around it, and the few bytes of
// its neighbours are not looked at.
#pragma once

#include "qk_norm_kernels.cuh"

namespace qk {

// What a thread reads and writes at once: a 16-byte vector or one element.
template <typename T, bool VEC>
struct Unit {
  using Raw = uint4;
  static constexpr int E = Vec16<T>::kElems;
  __device__ __forceinline__ static Raw load(const void* p, int64_t i) { return static_cast<const uint4*>(p)[i]; }
  __device__ __forceinline__ static Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ static void unpack(const Raw& r, float* f) { Vec16<T>::unpack_fresh(r, f); }
  __device__ __forceinline__ static Raw pack(const float* f) { return Vec16<T>::pack(f); }
  __device__ __forceinline__ static void store(void* p, int64_t i, const Raw& r) {
    __stcs(static_cast<uint4*>(p) + i, r);
  }
  // E values in 8 bits, as unit i of a row of bytes.
  __device__ __forceinline__ static void store8(void* p, int64_t i, const float* f, int qtype) {
    const uint32_t lo = quantise2(f[0], f[1], qtype) | quantise2(f[2], f[3], qtype) << 16;
    if constexpr (E == 8) {
      const uint32_t hi = quantise2(f[4], f[5], qtype) | quantise2(f[6], f[7], qtype) << 16;
      __stcs(static_cast<uint2*>(p) + i, make_uint2(lo, hi));
    } else {
      __stcs(static_cast<uint32_t*>(p) + i, lo);
    }
  }
};
template <typename T>
struct Unit<T, false> {
  using Raw = T;
  static constexpr int E = 1;
  __device__ __forceinline__ static Raw load(const void* p, int64_t i) { return static_cast<const T*>(p)[i]; }
  __device__ __forceinline__ static Raw zero() { return T(0.f); }
  __device__ __forceinline__ static void unpack(const Raw& r, float* f) { f[0] = float(r); }
  __device__ __forceinline__ static Raw pack(const float* f) { return T(f[0]); }
  __device__ __forceinline__ static void store(void* p, int64_t i, const Raw& r) { static_cast<T*>(p)[i] = r; }
  __device__ __forceinline__ static void store8(void* p, int64_t i, const float* f, int qtype) {
    static_cast<uint8_t*>(p)[i] = uint8_t(quantise(f[0], qtype));
  }
};

template <int OP, typename T, int THREADS, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(THREADS) norm_ring_kernel(const NormArgs a) {
  using U = Unit<T, VEC>;
  constexpr int E = U::E;
  constexpr int NW = THREADS / 32, WPG = TPR / 32, R = THREADS / TPR;
  static_assert(TPR % 32 == 0 && THREADS % TPR == 0 && NW <= 16, "row groups of whole warps");

  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  float* red = reinterpret_cast<float*>(smem + 512);             // [2][16] warp sums
  uint32_t* redm = reinterpret_cast<uint32_t*>(smem + 640);      // [2][16] warp maxima
  unsigned char* ring = smem + kSmemHeader;
  // 8-bit output by elements: maxima of 32 columns, a group's divisor and its reciprocal
  constexpr bool kBlocks = OP == kNormQuant && !VEC;
  __shared__ uint32_t blk[kBlocks ? 2 : 1][kBlocks ? 256 : 1];
  __shared__ float dens[kBlocks ? 2 : 1][kBlocks ? 256 : 1], invs[kBlocks ? 2 : 1][kBlocks ? 256 : 1];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = tid / TPR, l = tid % TPR;
  const int64_t M = a.M, N = a.N;
  const int NU = int(N / E);  // units of a row
  const int S = a.slots;
  const int nin = 1 + (a.r != nullptr) + (a.r2 != nullptr);  // inputs: x, r, r2 in this order
  const uint32_t slot_stride = uint32_t(nin) * a.slot_bytes;
  const int64_t n_local =
      a.num_items > int64_t(blockIdx.x) ? (a.num_items - 1 - blockIdx.x) / gridDim.x + 1 : 0;
  const uint32_t full0 = smem_addr(full), ring0 = smem_addr(ring);
  const unsigned char* in[3] = {static_cast<const unsigned char*>(a.x), static_cast<const unsigned char*>(a.r),
                                static_cast<const unsigned char*>(a.r2)};

  if (tid == 0) {
    for (int s = 0; s < S; ++s) mbar_init(full0 + 8 * s, 1);
    fence_mbar_init();
  }
  __syncthreads();

  // Bytes [off, off + bytes) of an item of an input; the copy is the 16-byte
  // aligned range around them, and `lead` is where they start in it.
  auto item_bytes = [&](int64_t item) { return min(int64_t(R), M - item * R) * N * int64_t(sizeof(T)); };
  auto lead_of = [&](int i, int64_t item) {
    return VEC ? 0u : uint32_t(reinterpret_cast<uintptr_t>(in[i]) + uint64_t(item * R * N * int64_t(sizeof(T)))) & 15u;
  };
  auto copy_item = [&](int64_t item, uint32_t dst, uint32_t bar, uint64_t policy, bool to_l2) {
    const int64_t bytes = item_bytes(item);
    uint32_t total = 0;
    for (int i = 0; i < nin; ++i) total += (lead_of(i, item) + uint32_t(bytes) + 15u) & ~15u;
    if (!to_l2) mbar_arrive_expect_tx(bar, total);
    for (int i = 0; i < nin; ++i) {
      const uint32_t lead = lead_of(i, item), n = (lead + uint32_t(bytes) + 15u) & ~15u;
      const unsigned char* src = in[i] + item * R * N * int64_t(sizeof(T)) - lead;
      for (uint32_t o = 0; o < n; o += 32768u) {
        if (to_l2)
          bulk_prefetch_l2(src + o, min(32768u, n - o));
        else
          bulk_copy_g2s(dst + uint32_t(i) * a.slot_bytes + o, src + o, min(32768u, n - o), bar, policy);
      }
    }
  };
  // The first item into L2 while the previous kernel of the stream finishes (a hint).
  if (tid == 0 && n_local > 0) copy_item(blockIdx.x, 0, 0, 0, true);
  grid_dependency_wait();
  allow_dependent_launch();

  uint64_t policy = 0;
  int64_t issued = 0;
  auto issue_next = [&]() {
    const int s = int(issued % S);
    copy_item(blockIdx.x + issued * gridDim.x, ring0 + uint32_t(s) * slot_stride, full0 + 8u * uint32_t(s), policy,
              false);
    ++issued;
  };
  if (tid == 0) {
    policy = l2_evict_first_policy();
    while (issued < S && issued < n_local) issue_next();
  }

  // The weight of this thread's columns stays in registers, as stored.
  typename U::Raw wv[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) wv[k] = l + k * TPR < NU ? U::load(a.w, l + k * TPR) : U::zero();
  float dw[OP == kAddNormBwd ? VPT * E : 1] = {};

  bool failed = false;
  int slot = 0;
  uint32_t phase = 0, bit = 0;
  int64_t q = 0;
  for (; q < n_local; ++q, bit ^= 1u) {
    const int64_t item = blockIdx.x + q * gridDim.x, row = item * R + g;
    float rs = 0.f;
    if (OP == kAddNormBwd && row < M) rs = __ldg(a.rstd + row);
    if (!mbar_wait<false>(full0 + 8u * uint32_t(slot), phase, a.timeout_ns)) {
      report_status(a.status, 5);
      failed = true;
    }
    const bool row_ok = row < M && !failed;
    const unsigned char* sb = ring + size_t(slot) * slot_stride + size_t(g) * size_t(N) * sizeof(T);
    typename U::Raw va[VPT], vb[VPT], vc[OP == kAddNormBwd ? VPT : 1];
    float acc = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int u = l + k * TPR;
      const bool ok = row_ok && u < NU;
      va[k] = ok ? U::load(sb + lead_of(0, item), u) : U::zero();
      vb[k] = ok && a.r != nullptr ? U::load(sb + a.slot_bytes + lead_of(1, item), u) : U::zero();
      if constexpr (OP == kAddNormBwd)
        vc[k] = ok && a.r2 != nullptr ? U::load(sb + 2 * a.slot_bytes + lead_of(2, item), u) : U::zero();
      float fa[E], fb[E];
      U::unpack(va[k], fa);
      U::unpack(vb[k], fb);
      if constexpr (OP == kAddNormBwd) {
        float fw[E];
        U::unpack(wv[k], fw);
#pragma unroll
        for (int e = 0; e < E; ++e) acc = fmaf(fb[e] * fw[e], fa[e], acc);
      } else {
        if (a.r != nullptr) {  // h, rounded as it is kept
#pragma unroll
          for (int e = 0; e < E; ++e) fa[e] += fb[e];
          va[k] = U::pack(fa);
          U::unpack(va[k], fa);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) acc = fmaf(fa[e], fa[e], acc);
      }
    }
    acc = group_sum<32>(acc);
    if (WPG > 1 && lane == 0) red[bit * 16 + warp] = acc;
    if (__syncthreads_or(failed)) break;  // also: every thread has read the slot
    if (tid == 0 && issued < n_local) issue_next();
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
    if constexpr (WPG > 1) {
      acc = 0.f;
#pragma unroll
      for (int i = 0; i < WPG; ++i) acc += red[bit * 16 + g * WPG + i];
    }
    const int64_t base = row * int64_t(NU);  // in units

    if constexpr (OP == kAddNormBwd) {
      if (!row_ok) continue;
      const float c = (acc * a.inv_n) * rs * rs * rs;  // in this order: rstd^3 alone may leave float32's range
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int u = l + k * TPR;
        if (u >= NU) continue;
        float fh[E], fd[E], fu[E], fw[E], o[E];
        U::unpack(va[k], fh);
        U::unpack(vb[k], fd);
        U::unpack(vc[k], fu);
        U::unpack(wv[k], fw);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          o[e] = fu[e] + fmaf(fh[e], -c, (rs * fd[e]) * fw[e]);
          dw[k * E + e] += (fd[e] * fh[e]) * rs;
        }
        U::store(a.y, base + u, U::pack(o));
      }
    } else {
      rs = 1.f / sqrtf(fmaf(acc, a.inv_n, a.eps));
      if (row_ok && l == 0 && a.rstd != nullptr) a.rstd[row] = rs;
      if (a.h != nullptr && row_ok) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
          if (l + k * TPR < NU) U::store(a.h, base + l + k * TPR, va[k]);
      }
      if constexpr (OP == kAddNorm) {
        if (!row_ok) continue;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const int u = l + k * TPR;
          if (u >= NU) continue;
          float f[E], fw[E];
          U::unpack(va[k], f);
          U::unpack(wv[k], fw);
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = (f[e] * rs) * fw[e];
          U::store(a.y, base + u, U::pack(f));
        }
      } else {
        // Largest |y| (times what EightBits has beside it) of each unit, as bits:
        // ordered like the numbers, infinity and NaN on top.
        const EightBits<T> eight(rs, a.qtype);
        float yv[VPT * E];
        uint32_t um[VPT], rowm = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          float* f = yv + k * E;
          float fw[E];
          U::unpack(va[k], f);
          U::unpack(wv[k], fw);
          um[k] = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            f[e] = (f[e] * eight.mul) * fw[e];
            um[k] = max(um[k], __float_as_uint(fabsf(f[e])));
          }
          rowm = max(rowm, um[k]);
        }
        if (a.group == 0) {
          rowm = __reduce_max_sync(0xffffffffu, rowm);
          if constexpr (WPG > 1) {
            if (lane == 0) redm[bit * 16 + warp] = rowm;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < WPG; ++i) rowm = max(rowm, redm[bit * 16 + g * WPG + i]);
          }
        } else if constexpr (VEC) {  // a group is 4 to 32 neighbouring lanes of one k
          const int lanes = a.group / E;
#pragma unroll
          for (int k = 0; k < VPT; ++k)
            for (int o = lanes / 2; o > 0; o >>= 1) um[k] = max(um[k], __shfl_xor_sync(0xffffffffu, um[k], o));
        } else {
          // A warp's 32 elements of one k lie in one group, and a group is 1, 2 or
          // 4 such blocks: block maxima, then a thread a group turns them into its
          // scale, its divisor and the reciprocal, which the row's threads read.
          const int per_row = (NU + 31) / 32, groups = int(a.groups);
#pragma unroll
          for (int k = 0; k < VPT; ++k) {
            um[k] = __reduce_max_sync(0xffffffffu, um[k]);
            if (lane == 0 && l + k * TPR < NU) blk[bit][g * per_row + (l + k * TPR) / 32] = um[k];
          }
          __syncthreads();
          for (int c = l; c < groups; c += TPR) {
            const int blocks = a.group / 32, first = c * blocks;
            uint32_t m = 0;
            for (int b = first; b < min(per_row, first + blocks); ++b) m = max(m, blk[bit][g * per_row + b]);
            float den;
            const float s = eight.scale(__uint_as_float(m), a.qtype, &den);
            if (row_ok) a.scale[row * a.groups + c] = s;
            dens[bit][g * groups + c] = den;
            invs[bit][g * groups + c] = eight.inverse(den);
          }
          __syncthreads();
        }
        if (!row_ok) continue;
        uint8_t* qrow = static_cast<uint8_t*>(a.y) + row * N;
        float* srow = a.scale + row * a.groups;
        float den = 0.f, inv = 0.f;
        const int shift = 31 - __clz(a.group);  // groups are powers of two
        if (a.group == 0) {
          const float s = eight.scale(__uint_as_float(rowm), a.qtype, &den);
          inv = eight.inverse(den);
          if (l == 0) srow[0] = s;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const int u = l + k * TPR;
          if (u >= NU) continue;
          if (!VEC && a.group != 0) {
            den = dens[bit][g * int(a.groups) + (u >> shift)];
            inv = invs[bit][g * int(a.groups) + (u >> shift)];
          } else if (a.group != 0) {
            const float s = eight.scale(__uint_as_float(um[k]), a.qtype, &den);
            inv = eight.inverse(den);
            if (((u * E) & (a.group - 1)) == 0) srow[(u * E) >> shift] = s;
          }
          float* f = yv + k * E;
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = quotient(f[e], den, inv);
          U::store8(qrow, u, f, a.qtype);
        }
      }
    }
  }

  if (q < n_local) {  // gave up: let the loads in flight land before leaving
    if (tid == 0)
      for (int64_t i = q + 1; i < issued; ++i) {
        if (++slot == S) {
          slot = 0;
          phase ^= 1u;
        }
        mbar_wait<false>(full0 + 8u * uint32_t(slot), phase, a.timeout_ns);
      }
    __syncthreads();
  }

  if constexpr (OP == kAddNormBwd) {
    // One partial row of dw a CTA: its row groups added in order, through the idle ring.
    float* out = a.dw_partial + int64_t(blockIdx.x) * N;
    float* sd = reinterpret_cast<float*>(ring);
    __syncthreads();
    for (int gg = 0; gg < R; ++gg) {
      if (g == gg) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int col = (l + k * TPR) * E + e;
            if (col < N) sd[col] = (gg == 0 ? 0.f : sd[col]) + dw[k * E + e];
          }
      }
      __syncthreads();
    }
    for (int64_t col = tid; col < N; col += THREADS) out[col] = sd[col];
  }
}

// ---------------------------------------------------------------------------
// The compiled row shapes: units a row, threads, threads a row, units a thread.
// ---------------------------------------------------------------------------
struct NormShape {
  int units, threads, row_threads, per_thread;
  const void* func;
};
struct NormTable {
  const NormShape* shapes;
  int count;
};

#define QK_NORM_SHAPE(OP, T, TH, TPR, VPT, VEC) \
  { TPR * VPT, TH, TPR, VPT, reinterpret_cast<const void*>(&norm_ring_kernel<OP, T, TH, TPR, VPT, VEC>) }
// Vectors: rows of up to 4096 (bf16 32768, fp32 16384 elements), 2048 in the
// backward.  The backward holds three inputs, the weight and dw in registers:
// two vectors a thread where a row is short (at four, one 256-thread CTA an SM
// fits: 32768 x 1024 bf16 ran at 65 % of the copy's rate).
#define QK_NORM_VECTOR_SHAPES(OP, T)                                                         \
  QK_NORM_SHAPE(OP, T, 256, 32, 1, true), QK_NORM_SHAPE(OP, T, 256, 32, 2, true),            \
      QK_NORM_SHAPE(OP, T, 256, 32, 4, true), QK_NORM_SHAPE(OP, T, 256, 64, 4, true),        \
      QK_NORM_SHAPE(OP, T, 128, 128, 4, true), QK_NORM_SHAPE(OP, T, 256, 256, 4, true),      \
      QK_NORM_SHAPE(OP, T, 512, 512, 4, true), QK_NORM_SHAPE(OP, T, 512, 512, 8, true)
#define QK_NORM_ELEMENT_SHAPES(OP, T)                                                        \
  QK_NORM_SHAPE(OP, T, 256, 32, 4, false), QK_NORM_SHAPE(OP, T, 256, 32, 8, false),          \
      QK_NORM_SHAPE(OP, T, 256, 32, 16, false), QK_NORM_SHAPE(OP, T, 256, 64, 16, false),    \
      QK_NORM_SHAPE(OP, T, 256, 128, 16, false), QK_NORM_SHAPE(OP, T, 256, 256, 16, false),  \
      QK_NORM_SHAPE(OP, T, 512, 512, 16, false)
#define QK_NORM_BWD_VECTOR_SHAPES(OP, T)                                                     \
  QK_NORM_SHAPE(OP, T, 256, 32, 1, true), QK_NORM_SHAPE(OP, T, 256, 32, 2, true),            \
      QK_NORM_SHAPE(OP, T, 256, 64, 2, true), QK_NORM_SHAPE(OP, T, 256, 128, 2, true),       \
      QK_NORM_SHAPE(OP, T, 128, 128, 4, true), QK_NORM_SHAPE(OP, T, 256, 256, 4, true),      \
      QK_NORM_SHAPE(OP, T, 512, 512, 4, true)

// Static shared memory of the kernels (the block maxima and scales of the 8-bit output), kept free beside the ring.
constexpr int kNormStaticSmem = 6144 + 16;

// Defined by the instantiation translation units: (operator, type) x (vectors, elements).
NormTable norm_shapes_add_f32(bool vec);
NormTable norm_shapes_add_bf16(bool vec);
NormTable norm_shapes_quant_f32(bool vec);
NormTable norm_shapes_quant_bf16(bool vec);
NormTable norm_shapes_bwd_f32(bool vec);
NormTable norm_shapes_bwd_bf16(bool vec);

}  // namespace qk
