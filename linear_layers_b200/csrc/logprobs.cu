// logprobs.cu — log-probabilities of given tokens, entropy and top
// alternatives of vocabulary-parallel logits, and their gradient.
//
//   z = scale·x,  M = max x,  S = Σ exp(scale·(x − M)),
//   U = Σ exp(scale·(x − M))·(x − M)
//   lse = scale·M + log S,  logprob = scale·(x_y − M) − log S,
//   entropy = log S − scale·U/S
//
// The sums run on differences to the maximum, so that neither a large common
// offset of a row nor a small entropy loses bits to the size of the logits.
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

// Descending value, then ascending index, as one unsigned order: 0 is "no
// entry" (NaN never enters).  +0 and −0 are the same value.
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t index) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<uint64_t>(o) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int32_t key_index(uint64_t key) {
  return static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key));
}

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

// One block per row: maximum, sums, then the alternatives one by one.
template <typename IT>
__global__ void __launch_bounds__(kRowThreads) logprobs_row_kernel(const LogprobsArgs a) {
  __shared__ float sf[kRowThreads / 32];
  __shared__ uint64_t sk[kRowThreads / 32];
  const int64_t t = blockIdx.x;
  const IT* row = static_cast<const IT*>(a.logits) + t * a.v;
  float m = -CUDART_INF_F;
  for (int64_t j = threadIdx.x; j < a.v; j += kRowThreads) m = fmaxf(m, to_f32(row[j]));
  m = block_reduce(m, sf, [](float p, float q) { return fmaxf(p, q); });
  if (m == -CUDART_INF_F) m = 0.0f;   // nothing but −inf (or NaN): S is 0 (or NaN)
  float s = 0.0f, u = 0.0f;
  const float sl = a.scale * kLog2e;
  for (int64_t j = threadIdx.x; j < a.v; j += kRowThreads) {
    const float d = to_f32(row[j]) - m;
    const float e = ex2_approx(d * sl);
    s += e;
    u = fmaf(e, fmaxf(d, -1e30f), u);
  }
  auto add = [](float p, float q) { return p + q; };
  s = block_reduce(s, sf, add);
  u = block_reduce(u, sf, add);
  const float log_s = logf(s);
  if (threadIdx.x == 0) {
    if (a.targets) {
      const int64_t y = a.targets[t];
      const bool ok = y >= 0 && y < a.v;
      if (!ok && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
      if (a.logprob) a.logprob[t] = ok ? fmaf(a.scale, to_f32(row[y]) - m, -log_s) : CUDART_NAN_F;
    }
    if (a.entropy) a.entropy[t] = log_s - a.scale * (u / s);
    if (a.lse) a.lse[t] = fmaf(a.scale, m, log_s);
  }
  uint64_t last = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    uint64_t best = 0;
    for (int64_t j = threadIdx.x; j < a.v; j += kRowThreads) {
      const float x = to_f32(row[j]);
      const uint64_t key = x == x ? rank_key(x, static_cast<uint32_t>(j)) : 0;
      if (key < last && key > best) best = key;
    }
    best = block_reduce(best, sk, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
    if (threadIdx.x == 0) {
      const int64_t o = t * a.top_k + k;
      a.top_idx[o] = best ? key_index(best) : -1;
      a.top_logprob[o] = best ? fmaf(a.scale, key_value(best) - m, -log_s) : CUDART_NAN_F;
    }
    last = best;
  }
}

template <typename IT, typename GT>
__global__ void __launch_bounds__(kRowThreads) logprobs_bwd_kernel(const LogprobsBwdArgs a) {
  const int64_t t = blockIdx.x;
  const IT* row = static_cast<const IT*>(a.logits) + t * a.v;
  GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
  const float g = a.dlogprob ? a.dlogprob[t] : 0.0f;
  const float e = a.dentropy ? a.dentropy[t] : 0.0f;
  if (g == 0.0f && e == 0.0f) {
    for (int64_t j = threadIdx.x; j < a.v; j += kRowThreads) put(out + j, 0.0f);
    return;
  }
  int64_t y = -1;
  float bad = 0.0f;
  if (g != 0.0f) {
    y = a.targets[t];
    if (y < 0 || y >= a.v) {
      bad = CUDART_NAN_F;
      if (threadIdx.x == 0 && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
    }
  }
  const float lse = a.lse[t];
  const float h = e != 0.0f ? a.entropy[t] : 0.0f;
  for (int64_t j = threadIdx.x; j < a.v; j += kRowThreads) {
    const float lp = fmaf(to_f32(row[j]), a.scale, -lse);
    const float p = ex2_approx(lp * kLog2e);
    const float d = (j == y ? g : 0.0f) - p * fmaf(e, fmaxf(lp, -1e30f) + h, g);
    put(out + j, a.scale * d + bad);
  }
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

// Combine of the per-slice statistics of the output-layer GEMM (slice k of
// row t at [k·T + t]): M = max m_k, w_k = exp(scale·(m_k − M)),
// S = Σ w_k·s_k, U = Σ w_k·(u_k + (m_k − M)·s_k).  32 tokens per block, one
// per lane; warp w reads slices w, w + 8, … and the eight partial results
// meet in warp order, so the sums do not depend on timing.
constexpr int kCombWarps = 8;

__global__ void __launch_bounds__(kCombWarps * 32)
    linear_logprobs_combine_kernel(const float* __restrict__ stat_m,
                                   const float* __restrict__ stat_s,
                                   const float* __restrict__ stat_u,
                                   const float* __restrict__ tgt_logit,
                                   const int64_t* __restrict__ targets, int64_t T, int64_t v,
                                   int nslices, float scale, float* __restrict__ logprob,
                                   float* __restrict__ entropy, float* __restrict__ lse,
                                   int32_t* dev_status) {
  __shared__ float part_m[kCombWarps][32];
  __shared__ float part_s[kCombWarps][32];
  __shared__ float part_u[kCombWarps][32];
  const int lane = threadIdx.x & 31;
  const int w = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const bool ok = t < T;
  float m = -CUDART_INF_F;
  if (ok) {
#pragma unroll 4
    for (int k = w; k < nslices; k += kCombWarps) m = fmaxf(m, stat_m[k * T + t]);
  }
  part_m[w][lane] = m;
  __syncthreads();
  float M = part_m[0][lane];
#pragma unroll
  for (int q = 1; q < kCombWarps; ++q) M = fmaxf(M, part_m[q][lane]);
  if (M == -CUDART_INF_F) M = 0.0f;   // nothing but −inf (or NaN) in the row
  float S = 0.0f, U = 0.0f;
  if (ok) {
#pragma unroll 4
    for (int k = w; k < nslices; k += kCombWarps) {
      const float d = stat_m[k * T + t] - M;
      const float f = ex2_approx(d * (scale * kLog2e));
      const float s = stat_s[k * T + t];
      S = fmaf(s, f, S);
      U = fmaf(f, fmaf(fmaxf(d, -1e30f), s, stat_u[k * T + t]), U);
    }
  }
  part_s[w][lane] = S;
  part_u[w][lane] = U;
  __syncthreads();
  if (w == 0 && ok) {
    S = 0.0f;
    U = 0.0f;
#pragma unroll
    for (int q = 0; q < kCombWarps; ++q) {
      S += part_s[q][lane];
      U += part_u[q][lane];
    }
    const float log_s = logf(S);
    if (targets) {
      const int64_t y = targets[t];
      const bool y_ok = y >= 0 && y < v;
      if (!y_ok && dev_status) atomicOr(dev_status, TP_DEVERR_RANGE);
      if (logprob)
        logprob[t] = y_ok ? fmaf(scale, tgt_logit[t] - M, -log_s) : CUDART_NAN_F;
    }
    if (entropy) entropy[t] = log_s - scale * (U / S);
    if (lse) lse[t] = fmaf(scale, M, log_s);
  }
}

tp_status last_error() { return cudaGetLastError() == cudaSuccess ? TP_OK : TP_ERR_CUDA; }

}  // namespace

tp_status logprobs_fwd_launch(const LogprobsArgs& a, tp_dtype dt, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.T);
  if (dt == TP_DTYPE_BF16)
    logprobs_row_kernel<__nv_bfloat16><<<grid, kRowThreads, 0, stream>>>(a);
  else
    logprobs_row_kernel<float><<<grid, kRowThreads, 0, stream>>>(a);
  note_launches(1);
  return last_error();
}

tp_status logprobs_bwd_launch(const LogprobsBwdArgs& a, tp_dtype dt, tp_dtype grad_dt,
                              cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.T);
  const bool ib = dt == TP_DTYPE_BF16, gb = grad_dt == TP_DTYPE_BF16;
  if (ib && gb)
    logprobs_bwd_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kRowThreads, 0, stream>>>(a);
  else if (ib)
    logprobs_bwd_kernel<__nv_bfloat16, float><<<grid, kRowThreads, 0, stream>>>(a);
  else if (gb)
    logprobs_bwd_kernel<float, __nv_bfloat16><<<grid, kRowThreads, 0, stream>>>(a);
  else
    logprobs_bwd_kernel<float, float><<<grid, kRowThreads, 0, stream>>>(a);
  note_launches(1);
  return last_error();
}

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

tp_status linear_logprobs_combine_launch(const float* stat_m, const float* stat_s,
                                         const float* stat_u, const float* tgt_logit,
                                         const int64_t* targets, int64_t T, int64_t v, float scale,
                                         float* logprob, float* entropy, float* lse,
                                         int32_t* dev_status, cudaStream_t stream) {
  const int nslices = static_cast<int>((v + kXentSlice - 1) / kXentSlice);
  linear_logprobs_combine_kernel<<<static_cast<unsigned>((T + 31) / 32), kCombWarps * 32, 0,
                                   stream>>>(stat_m, stat_s, stat_u, tgt_logit, targets, T, v,
                                             nslices, scale, logprob, entropy, lse, dev_status);
  note_launches(1);
  return last_error();
}

}  // namespace tpl
