// distill.cu — loss against a teacher's top entries and its gradient.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cstdint>

#include "internal.h"
#include "sm100_ptx.cuh"

namespace tpl {
namespace {

constexpr int kRowThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename V, typename F>
__device__ __forceinline__ V block_reduce(V x, V* sh, F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, off));
  if (lane == 0) sh[warp] = x;
  __syncthreads();
  x = sh[0];
  for (int w = 1; w < kRowThreads / 32; ++w) x = f(x, sh[w]);
  __syncthreads();
  return x;
}

// One block per row: log-sum-exp, the teacher's probabilities, the loss, then
// P·q everywhere and the teacher's entries over it.
template <typename IT, typename GT>
__global__ void __launch_bounds__(kRowThreads) distill_row_kernel(const DistillArgs a) {
  __shared__ float sf[kRowThreads / 32];
  __shared__ float sp[kDistillMaxK];
  __shared__ int32_t sid[kDistillMaxK];
  const int64_t t = blockIdx.x;
  const IT* row = static_cast<const IT*>(a.logits) + t * a.v;
  auto add = [](float p, float q) { return p + q; };
  auto max2 = [](float p, float q) { return fmaxf(p, q); };
  float m = -CUDART_INF_F;
  for (int64_t j = threadIdx.x; j < a.v; j += kRowThreads) m = fmaxf(m, to_f32(row[j]));
  m = block_reduce(m, sf, max2);
  if (m == -CUDART_INF_F) m = 0.0f;
  const float sl = a.scale * kLog2e;
  float s = 0.0f;
  for (int64_t j = threadIdx.x; j < a.v; j += kRowThreads)
    s += ex2_approx((to_f32(row[j]) - m) * sl);
  s = block_reduce(s, sf, add);
  const float log_s = logf(s);
  // the teacher's slots, one per thread
  const float w = a.weight ? a.weight[t] : 1.0f;
  int32_t id = -1;
  float tl = -CUDART_INF_F;
  if (threadIdx.x < a.K) {
    id = a.ids[t * a.K + threadIdx.x];
    if (id != -1) tl = a.teacher[t * a.K + threadIdx.x];
  }
  const bool bad = id < -1 || id >= a.v;
  const float any_bad = block_reduce(bad ? 1.0f : 0.0f, sf, max2);
  if (bad) tl = -CUDART_INF_F;
  float tm = 0.0f, log_ts = 0.0f;
  if (a.renormalize) {
    tm = block_reduce(tl, sf, max2);
    if (tm == -CUDART_INF_F) tm = 0.0f;
    const float ts = block_reduce(expf(tl - tm), sf, add);
    log_ts = ts == 0.0f ? 0.0f : logf(ts);
  }
  const float lp = tl - tm - log_ts;
  const float p = id == -1 || bad ? 0.0f : expf(lp);
  const float P = block_reduce(p, sf, add);
  float term = 0.0f, xk = 0.0f;
  if (p != 0.0f) {
    xk = to_f32(row[id]);
    term = p * (lp - fmaf(a.scale, xk - m, -log_s));
  }
  const float loss = block_reduce(term, sf, add);
  const bool dead = w == 0.0f || (P == 0.0f && any_bad == 0.0f);
  const bool invalid = !dead && any_bad != 0.0f;
  if (threadIdx.x == 0) {
    a.loss[t] = dead ? 0.0f : invalid ? CUDART_NAN_F : w * loss;
    if (a.lse) a.lse[t] = fmaf(a.scale, m, log_s);
    if (invalid && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
  }
  if (!a.dlogits) return;
  if (threadIdx.x < a.K) {
    sid[threadIdx.x] = id;
    sp[threadIdx.x] = p;
  }
  __syncthreads();
  GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
  const float c = a.grad_scale * w * a.scale;
  const float f = invalid ? CUDART_NAN_F : c;
  float patch = 0.0f;
  bool first = threadIdx.x < a.K && id >= 0 && !bad;
  if (first) {
    float sum = 0.0f;
    for (int k = 0; k < a.K; ++k)
      if (sid[k] == id) {
        if (k < static_cast<int>(threadIdx.x)) first = false;
        sum += sp[k];
      }
    patch = P * ex2_approx((to_f32(row[id]) - m) * sl) / s - sum;
  }
  __syncthreads();
  for (int64_t j = threadIdx.x; j < a.v; j += kRowThreads) {
    const float q = ex2_approx((to_f32(row[j]) - m) * sl) / s;
    put(out + j, dead ? 0.0f : f * (P * q));
  }
  __syncthreads();
  if (first && !dead) put(out + id, f * patch);
}

tp_status last_error() { return cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA; }

}  // namespace

tp_status distill_launch(const DistillArgs& a, tp_dtype dt, tp_dtype grad_dt, float* loss_sum,
                         cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.T);
  const bool ib = dt == TP_DTYPE_BF16, gb = grad_dt == TP_DTYPE_BF16;
  if (ib && gb)
    distill_row_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kRowThreads, 0, stream>>>(a);
  else if (ib)
    distill_row_kernel<__nv_bfloat16, float><<<grid, kRowThreads, 0, stream>>>(a);
  else if (gb)
    distill_row_kernel<float, __nv_bfloat16><<<grid, kRowThreads, 0, stream>>>(a);
  else
    distill_row_kernel<float, float><<<grid, kRowThreads, 0, stream>>>(a);
  note_launches(1);
  if (tp_status st = last_error()) return st;
  return loss_sum ? loss_sum_launch(a.loss, a.T, loss_sum, stream) : TP_OK;
}

}  // namespace tpl
