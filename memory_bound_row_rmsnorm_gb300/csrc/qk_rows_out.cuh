// qk_rows_out.cuh -- the way of a product's rows from registers to memory.
#pragma once

#include "qk_device.cuh"

namespace qk {

constexpr int kOutBytes = 32 * 128;  // an epilogue warp's 32 rows of 128 bytes on their way out

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

}  // namespace qk
