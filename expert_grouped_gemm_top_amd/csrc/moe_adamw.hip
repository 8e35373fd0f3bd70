// moe_adamw.hip -- an AdamW step over many tensors in one launch, with moments
// of 32 bits or of 8.
//
//   t = step + 1,  g' = grad_scale g
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr decay) - lr m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps)
//
// HBM-bound: every element of every tensor is read once and written once (22
// bytes of bf16 weight, gradient and 32-bit moments, 28 with an fp32 master, 10
// with 8-bit moments).
//
// What is held in fewer bits than it changes by is rounded up or down by a hash
// of the element's place, the step and the seed, up with the probability of what
// is left over: bf16 weights without a master (a step of 1e-5 beside a weight of
// 0.02 is a tenth of half a bf16 step: rounded to nearest it would never come
// about), and 8-bit moments (v moves by a thousandth of its distance to g^2, a
// sixtieth of a code's half step: to nearest it would stand still).  So the
// expected values are the exact ones.
#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

#include "moe_common.h"
#include "moe_launch.h"
#include "moe_rows.h"

namespace moe {

namespace {

// ---- the hash ------------------------------------------------------------------

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x85ebca77u;
  x = (x ^ (x >> 15)) * 0xc2b2ae3du;
  return x ^ (x >> 16);
}

// ---- moments in 8 bits ------------------------------------------------------------

// Blocks of 256 elements share a power-of-two scale.  m: E4M3 (bias 7, largest
// 448).  v, which has no sign and twice the range: 5 bits of exponent, 3 of
// mantissa, code c = (8 + c % 8) 2^(c / 8 - 34), 0 zero, 254 the largest, 1.75.
// Both keep NaN (0x7f, 255) for elements that are not finite.  A root of v that
// was rounded to zero would divide by eps alone: what is not zero stays so.
//
// m and v are formed in 64 bits, so that the code and the scale of every element
// are those of the formula: in 32 bits one in some millions would fall on the
// other side of a border, and differ by a whole code.
constexpr int kMaxM = 126, kMaxV = 254;

__device__ __forceinline__ float value_m(uint32_t code) { return __builtin_amdgcn_cvt_f32_fp8((int)code, 0); }
__device__ __forceinline__ float value_v(uint32_t code) {
  if (code == 255) return __builtin_nanf("");
  return code == 0 ? 0.0f : __uint_as_float((code + ((127 - 31) << 3)) << 20);
}

// 2^e as a double.
__device__ __forceinline__ double pow2(int e) { return __hiloint2double((e + 1023) << 20, 0); }

// Exponent of the smallest power of two s with top <= 1.75 2^up s: 448 = 1.75 2^8.
__device__ __forceinline__ int scale_exponent(float top, int up) {
  const uint32_t bits = __float_as_uint(top);
  const int e = (int)(bits >> 23) - 127 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0) - up;
  return min(max(e, -126), 127);  // subnormal tops lie below the first
}

// The size of a finite value as fp32, for the scale.
__device__ __forceinline__ float size_of(double a) {
  const float f = fabsf((float)a);
  return a - a == 0.0 ? fminf(f, 3.402823466e38f) : 0.0f;
}

// Codes of a >= 0 by their exponent and three bits of mantissa, from 2^least on in
// steps of an eighth of the binade, below in those of that binade (codes from -8
// on).  Rounded up for the share (h + 1/3) / 2^16 of what is left over (the third
// keeps the border off values that short binary codes and gradients add up to).
__device__ __forceinline__ int eighths(double a, int least, uint32_t h) {
  const bool small = a < pow2(least);
  const uint64_t b = (uint64_t)__double_as_longlong(small ? a + pow2(least) : a) + (((uint64_t)h << 33) + 0xaaaaaaaau);
  return (int)(b >> 49) - ((1023 + least) << 3) - (small ? 8 : 0);
}
__device__ __forceinline__ uint32_t code_m(double a, uint32_t h) {
  if (a - a != 0.0) return 0x7f;
  const int c = min(eighths(fabs(a), -6, h) + 8, kMaxM);  // 2^-6 has code 8
  return (uint32_t)c | (a < 0.0 ? 0x80u : 0u);
}
__device__ __forceinline__ uint32_t code_v(double a, uint32_t h) {
  if (a - a != 0.0) return 255;
  if (a == 0.0) return 0;
  return (uint32_t)min(max(eighths(a, -31, h), 1), kMaxV);
}

// ---- the step ----------------------------------------------------------------------

struct AdamwArgs {
  const AdamwEntry* entries;
  const int64_t* starts;  // first chunk of each tensor, and their number behind the last
  int n;
  int64_t chunks;
  int32_t* counter;  // {steps done, workgroups done}
  const float* lr;
  const float* grad_scale;
  double beta1, beta2, log_beta1, log_beta2;
  float eps;
  uint32_t seed;
};

// What all elements share.
struct Shared {
  double gs;
  float step1, inv_root2, lr;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t key;
};

__device__ __forceinline__ float updated(float p, float keep, float m, float v, const Shared& sh, float eps) {
  return p * keep - sh.step1 * (m / (sqrtf(v) * sh.inv_root2 + eps));
}

// bf16 of p, rounded by 16 of the hash's bits.
__device__ __forceinline__ uint32_t dithered(float p, uint32_t r) {
  const uint32_t bits = __float_as_uint(p);
  if ((bits & 0x7f800000u) == 0x7f800000u) return f2bf(p);
  return (bits + ((r * 0x9e3779b1u) >> 16)) >> 16;
}

template <typename T, bool MASTER, bool SMALL>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwArgs g) {
  __shared__ Shared s_sh;
  const int tid = threadIdx.x;
  if (tid == 0) {
    const int t = g.counter[0] + 1;
    const double lr = *g.lr;
    s_sh.gs = g.grad_scale != nullptr ? (double)*g.grad_scale : 1.0;
    s_sh.lr = (float)lr;
    s_sh.step1 = (float)(lr / -expm1(t * g.log_beta1));
    s_sh.inv_root2 = (float)(1.0 / sqrt(-expm1(t * g.log_beta2)));
    s_sh.key = mix32(mix32((uint32_t)t) + g.seed);
  }
  __syncthreads();
  const Shared sh = s_sh;
  const float b1 = (float)g.beta1, a1 = (float)(1.0 - g.beta1), b2 = (float)g.beta2, a2 = (float)(1.0 - g.beta2);
  const float gs = (float)sh.gs;
  int i = 0;
  int64_t from = 0, to = 0;  // chunks of tensor i
  AdamwEntry e{};
  for (int64_t chunk = blockIdx.x; chunk < g.chunks; chunk += gridDim.x) {
    if (chunk >= to) {
      int hi = g.n;  // the last tensor that begins at or before the chunk: those before it are empty or done
      while (hi - i > 1) {
        const int mid = (i + hi) >> 1;
        if (g.starts[mid] <= chunk) i = mid; else hi = mid;
      }
      from = g.starts[i];
      to = g.starts[i + 1];
      e = g.entries[i];
    }
    const int64_t at = (chunk - from) * kAdamwChunk + 8 * tid;  // of this thread's eight elements
    const int live = (int)min((int64_t)8, max((int64_t)0, e.numel - at));
    const float keep = (float)(1.0 - (double)sh.lr * e.decay);
    const uint64_t place = (uint64_t)e.first * kAdamwBlock + (uint64_t)at;
    float p[8], gr[8];
    T* param = (T*)e.param + at;
    const T* grad = (const T*)e.grad + at;
    if (live == 8) {
      load8(grad, gr);
      if (MASTER) load8(e.master + at, p);
      else load8(param, p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gr[j] = j < live ? load1(grad + j) : 0.0f;
        p[j] = j < live ? (MASTER ? e.master[at + j] : load1(param + j)) : 0.0f;
      }
    }
    uint32_t r[8];
    if (SMALL || (!MASTER && sizeof(T) == 2)) {
      const uint32_t key = sh.key ^ mix32((uint32_t)(place >> 32)) * (uint32_t)((place >> 32) != 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = mix32(((uint32_t)place + j) ^ key);
    }
    if (!SMALL) {
      float m[8], v[8];
      float *mp = (float*)e.m + at, *vp = (float*)e.v + at;
      if (live == 8) {
        load8(mp, m);
        load8(vp, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[j] = j < live ? mp[j] : 0.0f;
          v[j] = j < live ? vp[j] : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gj = gr[j] * gs;
        m[j] = b1 * m[j] + a1 * gj;
        v[j] = b2 * v[j] + a2 * gj * gj;
        p[j] = updated(p[j], keep, m[j], v[j], sh, g.eps);
      }
      if (live == 8) {
        store8(mp, m);
        store8(vp, v);
      } else {
        for (int j = 0; j < live; ++j) {
          mp[j] = m[j];
          vp[j] = v[j];
        }
      }
    } else {
      uint8_t *mp = (uint8_t*)e.m + at, *vp = (uint8_t*)e.v + at;
      uint32_t mc[2] = {}, vc[2] = {};
      if (live == 8) {
        const u32x2 a = *(const u32x2*)mp, b = *(const u32x2*)vp;
        mc[0] = a[0], mc[1] = a[1], vc[0] = b[0], vc[1] = b[1];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          mc[j >> 2] |= (j < live ? (uint32_t)mp[j] : 0u) << (8 * (j & 3));
          vc[j >> 2] |= (j < live ? (uint32_t)vp[j] : 0u) << (8 * (j & 3));
        }
      }
      const int64_t block = at / kAdamwBlock;
      const double ms = live > 0 ? (double)e.m_scale[block] : 0.0, vs = live > 0 ? (double)e.v_scale[block] : 0.0;
      double m[8], v[8];
      float top_m = 0.0f, top_v = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double gj = (double)gr[j] * sh.gs;
        m[j] = g.beta1 * ((double)value_m((mc[j >> 2] >> (8 * (j & 3))) & 255) * ms) + (1.0 - g.beta1) * gj;
        v[j] = g.beta2 * ((double)value_v((vc[j >> 2] >> (8 * (j & 3))) & 255) * vs) + (1.0 - g.beta2) * gj * gj;
        p[j] = updated(p[j], keep, (float)m[j], (float)v[j], sh, g.eps);
        top_m = fmaxf(top_m, size_of(m[j]));
        top_v = fmaxf(top_v, size_of(v[j]));
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {  // the 32 lanes of a block
        top_m = fmaxf(top_m, __shfl_xor(top_m, o, kWave));
        top_v = fmaxf(top_v, __shfl_xor(top_v, o, kWave));
      }
      const int em = scale_exponent(top_m, 8), ev = scale_exponent(top_v, 0);
      const double im = pow2(-em), iv = pow2(-ev);
      mc[0] = mc[1] = vc[0] = vc[1] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mc[j >> 2] |= code_m(m[j] * im, r[j] & 0xffffu) << (8 * (j & 3));
        vc[j >> 2] |= code_v(v[j] * iv, r[j] >> 16) << (8 * (j & 3));
      }
      if (live == 8) {
        *(u32x2*)mp = u32x2{mc[0], mc[1]};
        *(u32x2*)vp = u32x2{vc[0], vc[1]};
      } else {
        for (int j = 0; j < live; ++j) {
          mp[j] = (uint8_t)(mc[j >> 2] >> (8 * (j & 3)));
          vp[j] = (uint8_t)(vc[j >> 2] >> (8 * (j & 3)));
        }
      }
      if ((tid & 31) == 0 && live > 0) {
        e.m_scale[block] = (float)pow2(em);
        e.v_scale[block] = (float)pow2(ev);
      }
    }
    if (MASTER) {
      if (live == 8) {
        store8(e.master + at, p);
        store8(param, p);
      } else {
        for (int j = 0; j < live; ++j) {
          e.master[at + j] = p[j];
          store1(param + j, p[j]);
        }
      }
    } else if constexpr (sizeof(T) == 2) {
      uint32_t q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = dithered(p[j], r[j]);
      if (live == 8) *(u32x4*)param = u32x4{q[0] | q[1] << 16, q[2] | q[3] << 16, q[4] | q[5] << 16, q[6] | q[7] << 16};
      else
        for (int j = 0; j < live; ++j) param[j] = (T)q[j];
    } else {
      if (live == 8) store8(param, p);
      else
        for (int j = 0; j < live; ++j) store1(param + j, p[j]);
    }
  }
  // The last workgroup to get here counts the step: every one has read the counter.
  if (tid == 0 && (uint32_t)atomicAdd((uint32_t*)g.counter + 1, 1u) == gridDim.x - 1) {
    g.counter[1] = 0;
    g.counter[0] += 1;
  }
}

// The moments that codes stand for.  HBM-bound: 2 bytes read, 8 written an element.
__global__ __launch_bounds__(256) void adamw_moments_kernel(int64_t numel, const uint8_t* __restrict__ m,
                                                            const uint8_t* __restrict__ v,
                                                            const float* __restrict__ m_scale,
                                                            const float* __restrict__ v_scale, float* __restrict__ m_out,
                                                            float* __restrict__ v_out) {
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; at < numel; at += (int64_t)gridDim.x * 2048) {
    const double ms = (double)m_scale[at / kAdamwBlock], vs = (double)v_scale[at / kAdamwBlock];
    const int live = (int)min((int64_t)8, numel - at);
    float a[8], b[8];
    if (live == 8) {
      const u32x2 mc = *(const u32x2*)(m + at), vc = *(const u32x2*)(v + at);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = (float)((double)value_m((mc[j >> 2] >> (8 * (j & 3))) & 255) * ms);
        b[j] = (float)((double)value_v((vc[j >> 2] >> (8 * (j & 3))) & 255) * vs);
      }
      store8(m_out + at, a);
      store8(v_out + at, b);
    } else {
      for (int j = 0; j < live; ++j) {
        m_out[at + j] = (float)((double)value_m(m[at + j]) * ms);
        v_out[at + j] = (float)((double)value_v(v[at + j]) * vs);
      }
    }
  }
}

struct Plan {
  uint32_t magic;
  int n, esize, small, master;
  int64_t chunks;
};
constexpr uint32_t kPlanMagic = 0x61646d77u;
constexpr size_t kPlanHead = 64;
static_assert(sizeof(Plan) <= kPlanHead, "the plan's head");

size_t starts_offset(int n) { return kPlanHead + (size_t)n * sizeof(AdamwEntry); }

}  // namespace

size_t adamw_plan_bytes(int n) { return starts_offset(n) + ((size_t)n + 1) * sizeof(int64_t); }

void adamw_make_plan(int n, const AdamwEntry* entries, int esize, bool small, bool master, void* plan) {
  Plan h{kPlanMagic, n, esize, small, master, 0};
  int64_t block = 0;
  for (int i = 0; i < n; ++i) {
    AdamwEntry e = entries[i];
    e.first = block;
    block += (e.numel + kAdamwBlock - 1) / kAdamwBlock;
    memcpy((char*)plan + kPlanHead + i * sizeof e, &e, sizeof e);
    memcpy((char*)plan + starts_offset(n) + i * sizeof(int64_t), &h.chunks, sizeof h.chunks);
    h.chunks += (e.numel + kAdamwChunk - 1) / kAdamwChunk;
  }
  memcpy((char*)plan + starts_offset(n) + n * sizeof(int64_t), &h.chunks, sizeof h.chunks);
  memset(plan, 0, kPlanHead);
  memcpy(plan, &h, sizeof h);
}

bool adamw_is_plan(const void* plan) {
  uint32_t magic;
  memcpy(&magic, plan, sizeof magic);
  return magic == kPlanMagic;
}

hipError_t launch_adamw(const void* plan, const void* plan_device, const AdamwStep& a, hipStream_t stream) {
  Plan h;
  memcpy(&h, plan, sizeof h);
  AdamwArgs g{};
  g.entries = (const AdamwEntry*)((const char*)plan_device + kPlanHead);
  g.starts = (const int64_t*)((const char*)plan_device + starts_offset(h.n));
  g.n = h.n;
  g.chunks = h.chunks;
  g.counter = a.counter;
  g.lr = a.lr;
  g.grad_scale = a.grad_scale;
  g.beta1 = a.beta1;
  g.beta2 = a.beta2;
  g.log_beta1 = a.beta1 > 0.0 ? log(a.beta1) : -__builtin_inf();
  g.log_beta2 = a.beta2 > 0.0 ? log(a.beta2) : -__builtin_inf();
  g.eps = (float)a.eps;
  g.seed = a.seed;
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(h.chunks, 2048))), block(256);
  auto run = [&](auto kernel) {
    MOE_LAUNCH(kernel, grid, block, 0, stream, g);
    return hipGetLastError();
  };
  if (h.esize == 4) return h.small ? run(adamw_kernel<float, false, true>) : run(adamw_kernel<float, false, false>);
  if (h.master)
    return h.small ? run(adamw_kernel<uint16_t, true, true>) : run(adamw_kernel<uint16_t, true, false>);
  return h.small ? run(adamw_kernel<uint16_t, false, true>) : run(adamw_kernel<uint16_t, false, false>);
}

hipError_t launch_adamw_moments(int64_t numel, const uint8_t* m, const uint8_t* v, const float* m_scale,
                                const float* v_scale, float* m_out, float* v_out, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>((numel + 2047) / 2048, 8192));
  MOE_LAUNCH(adamw_moments_kernel, grid, dim3(256), 0, stream, numel, m, v, m_scale, v_scale, m_out, v_out);
  return hipGetLastError();
}

}  // namespace moe
