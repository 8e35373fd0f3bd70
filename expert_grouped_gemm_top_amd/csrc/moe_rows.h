// moe_rows.h -- device helpers of the row-wise kernels: runs of eight
// neighbouring elements of an fp32 or bf16 row as fp32 values.
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
// The same, past the caches where `stream` (rows that no cache would hold until they are read again).
__device__ __forceinline__ void store8(float* p, const float (&v)[8], bool stream) {
  if (!stream) return store8(p, v);
  __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4*)p);
  __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, (f32x4*)(p + 4));
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], bool stream) {
  if (!stream) return store8(p, v);
  __builtin_nontemporal_store(u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]),
                                    pack_bf2(v[6], v[7])}, (u32x4*)p);
}

// Eight elements as they lie in memory, to be converted later (a load in flight).
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  f32x4 lo, hi;
  __device__ __forceinline__ void load(const float* p) {
    lo = *(const f32x4*)p;
    hi = *(const f32x4*)(p + 4);
  }
  __device__ __forceinline__ float get(int j) const { return j < 4 ? lo[j] : hi[j - 4]; }
};
template <>
struct Raw8<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *(const u32x4*)p; }
  __device__ __forceinline__ float get(int j) const { return (j & 1) ? bf_hi(v[j >> 1]) : bf_lo(v[j >> 1]); }
};
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)f2bf(v); }

}  // namespace moe
