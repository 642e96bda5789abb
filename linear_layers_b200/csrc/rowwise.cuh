// rowwise.cuh — reading rows of logits and adding up their softmax sums, for
// the kernels of logprobs.cu and distill.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "row_split.h"
#include "sm100_ptx.cuh"

namespace tpl {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -1e30f;   // stands for what lies below it in products with a zero probability

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Logits are read once: 16-byte units that do not stay in L1.
__device__ __forceinline__ uint4 ld_unit(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename IT>
struct Unit;   // the elements of 16 bytes
template <>
struct Unit<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kMinusInf = 0xff800000u;
  static __device__ __forceinline__ void unpack(uint4 w, float* x) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
};
template <>
struct Unit<__nv_bfloat16> {
  static constexpr int kN = 8;
  static constexpr uint32_t kMinusInf = 0xff80ff80u;
  static __device__ __forceinline__ void unpack(uint4 w, float* x) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(q[i] << 16);
      x[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// N consecutive gradient elements at p (N·sizeof aligned to 8 bytes or more)
template <int N>
__device__ __forceinline__ void put_unit(float* p, const float* x) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    __stcs(reinterpret_cast<float4*>(p) + i,
           make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}
template <int N>
__device__ __forceinline__ void put_unit(__nv_bfloat16* p, const float* x) {
  if constexpr (N == 4)
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])));
  else
    __stcs(reinterpret_cast<uint4*>(p),
           make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7])));
}

template <typename IT>
using RowShape = RowSplit<Unit<IT>::kN>;

// Running softmax sums of one thread over raw logits: s = Σ e, u = Σ e·(x − r)
// with e = exp(scale·(x − r)).  Any reference r gives the same sums but for
// their rounding: with r a distance δ = scale·(M − r) below the row's maximum,
// entropy = log S − scale·U/S is a difference of two numbers of size δ, whose
// rounding errors it keeps.  r moves when a logit exceeds it by more than
// 2 in log2 units, so δ < 1.4; within 8 (δ < 5.6) the entropies of rows whose two
// highest logits lie 5 apart were off by up to 5.0e-6 of their size, within 2 by
// 6.7e-7, at r = M by 5.5e-7.  A thread that has seen no logit above −inf keeps
// r = 0 with the threshold at −inf, unless its warp started at one.
struct RowSums {
  float ref = 0.0f, above = -INFINITY;
  float2 s = {0.0f, 0.0f}, u = {0.0f, 0.0f};

  // A first reference for the whole warp, the largest of its lanes' x: the
  // steps behind it move references less often than from one of each lane.
  template <int N>
  __device__ __forceinline__ void start(const float (&x)[N], float tau) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (m > -INFINITY) {
      ref = m;
      above = m + tau;
    }
  }

  template <int N, bool kEntropy>
  __device__ __forceinline__ float add(const float (&x)[N], float sl, float tau) {
    float mx = max3f(fmaxf(x[0], x[1]), x[2], x[3]);
#pragma unroll
    for (int i = 4; i < N; i += 4) mx = max3f(max3f(mx, x[i], x[i + 1]), x[i + 2], x[i + 3]);
    if (mx > above) {
      const float dm = above == -INFINITY ? 0.0f : max_nan(ref - mx, kLowest);
      const float al = ex2_approx(dm * sl);
      if (kEntropy)
        u = make_float2(al * fmaf(dm, s.x, u.x), al * fmaf(dm, s.y, u.y));
      s = make_float2(al * s.x, al * s.y);
      ref = mx;
      above = mx + tau;
    }
    const float2 nr = make_float2(-ref, -ref), sl2 = make_float2(sl, sl);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float2 d = __fadd2_rn(make_float2(x[i], x[i + 1]), nr);
      if (kEntropy) d = make_float2(max_nan(d.x, kLowest), max_nan(d.y, kLowest));
      const float2 y = __fmul2_rn(d, sl2);
      const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
      s = __fadd2_rn(s, e);
      if (kEntropy) u = __ffma2_rn(e, d, u);
    }
    return mx;
  }
  // one element (the row's edges)
  template <bool kEntropy>
  __device__ __forceinline__ void add1(float x, float sl, float tau) {
    const float q[4] = {x, -INFINITY, -INFINITY, -INFINITY};
    add<4, kEntropy>(q, sl, tau);
  }
};

// The sums of several threads, on a common reference: m = −inf where nothing
// above −inf was seen.
struct Sums {
  float m, s, u;
};

// The sum of n <= 32 sums, lane i bringing the i-th (any value past n): the
// shuffles of a whole warp, the same order and result in every caller.
__device__ __forceinline__ Sums join_sums(int n, Sums q, float sl) {
  if (static_cast<int>(threadIdx.x & 31) >= n) q = Sums{-INFINITY, 0.0f, 0.0f};
  float m = q.m;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float d = max_nan(q.m - (m == -INFINITY ? 0.0f : m), kLowest);
  const float f = ex2_approx(d * sl);
  float s = q.s * f, u = f * fmaf(d, q.s, q.u);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, off);
    u += __shfl_xor_sync(0xffffffffu, u, off);
  }
  return Sums{m, s, u};
}

// The sums of a warp's threads, on a common reference.
__device__ __forceinline__ Sums warp_sums(const RowSums& r, float sl) {
  return join_sums(32,
                   Sums{r.above == -INFINITY ? -INFINITY : r.ref, r.s.x + r.s.y, r.u.x + r.u.y},
                   sl);
}

}  // namespace tpl
