// tf32.cuh — fp32 products on the tensor cores in three passes of tf32.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace cp {

// x = hi + lo: hi rounded to tf32's 11 bits (half away from zero), so that lo has
// either sign and what the multiplier does not read of it (2^-22 of x at most)
// averages out over a sum.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// d += a b, m16n8k8: a[e] is row g + 8 (e % 2), column t + 4 (e / 2); b0, b1 rows
// t, t + 4, column g; d[e] row g + 8 (e / 2), column 2 t + e % 2 (g = lane / 4, t = lane % 4)
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// big += hi hi', small += hi lo' + lo hi'; lo lo' (2^-24) is left out. The
// accumulators' additions truncate, which adds up along a long sum (3.9e-6 of dq
// over 700 keys), so callers start big anew every few steps and add it up by
// rounding additions (4e-7).
__device__ __forceinline__ void mma3_tf32(float (&big)[4], float (&small)[4], const uint32_t (&ah)[4],
                                          const uint32_t (&al)[4], const uint32_t (&bh)[2], const uint32_t (&bl)[2]) {
  mma_tf32(small, al, bh[0], bh[1]);
  mma_tf32(big, ah, bh[0], bh[1]);
  mma_tf32(small, ah, bl[0], bl[1]);
}

}  // namespace cp
