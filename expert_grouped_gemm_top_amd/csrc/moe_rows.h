// moe_rows.h -- device helpers of the row-wise kernels: runs of eight
// neighbouring elements of an fp32 or bf16 row as fp32 values, and sums of
// per-workgroup column partials.
#pragma once

#include "moe_common.h"

namespace moe {

// Eight elements at p (16-byte aligned) as fp32.
__device__ __forceinline__ void load8(const float* __restrict__ p, float (&v)[8]) {
  const f32x4 lo = *(const f32x4*)p, hi = *(const f32x4*)(p + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = lo[j];
    v[4 + j] = hi[j];
  }
}
__device__ __forceinline__ void load8(const uint16_t* __restrict__ p, float (&v)[8]) {
  const u32x4 r = *(const u32x4*)p;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf_lo(r[j]);
    v[2 * j + 1] = bf_hi(r[j]);
  }
}
// The same values rounded once to the element type.
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *(u32x4*)p = u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])};
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)f2bf(v); }

}  // namespace moe
