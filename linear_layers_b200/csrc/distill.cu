// distill.cu — loss of softmax(scale·logits) against a teacher's top entries,
// and its gradient, in one pass over the logits.
//
//   p_k: the teacher's probabilities on K listed tokens, P = Σ p_k,
//   C = Σ p_k·log p_k,  r = max x,  S = Σ exp(scale·(x − r)),
//   A = Σ p_k·(x_{id_k} − r)
//   loss = w·(C − scale·A + P·log S)
//   dlogits_j = grad_scale·w·scale·(P·exp(scale·(x_j − r))/S − Σ_{k: id_k = j} p_k)
//
// Every logit is needed twice, once for S and once for the gradient, and a
// row of 50304 fp32 logits (201 KB) is wider than two SMs can buffer: so a
// cluster of up to eight blocks holds one row, each block its slice in shared
// memory.  HBM sees each logit read once and each gradient written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "rowwise.cuh"
#include "sm100_ptx.cuh"

namespace tpl {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxSlices = 8;
constexpr int kSlots = kDistillMaxK / 32;   // teacher slots per lane

// 1-D bulk copy global -> this CTA's shared memory, completion counted in
// bytes on `bar` (16-byte aligned addresses, size a multiple of 16).
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* gsrc, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(gsrc)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// Persistent clusters of `slices` blocks; cluster c handles rows c, c + C, …
// Block r of a cluster owns units [r·per, (r+1)·per) of each row, staged by
// bulk copies `nbuf` rows ahead, block 0 also the row's edges.  Per row:
//   1. the last warp turns the teacher's slots into probabilities (loaded a
//      row ahead) while the others wait for the slice;
//   2. every thread adds up its units; the block's (r, S, A, P of its own
//      tokens) goes to every block of the cluster as one 16-byte asynchronous
//      store counted on the receiver's barrier;
//   3. the blocks combine the records in slice order, write P·q over their
//      slice and, behind a block barrier, the listed tokens over that; the
//      buffer is refilled at the same barrier.
template <typename IT, typename GT>
__global__ void __launch_bounds__(kMaxThreads, 1)
    distill_kernel(const DistillArgs a, int slices, int per, int nbuf, uint32_t buf_stride,
                   uint64_t wait_ns) {
  constexpr int kN = Unit<IT>::kN;
  extern __shared__ __align__(128) uint8_t buffers[];
  __shared__ __align__(16) float rec[2][kMaxSlices][4];   // [row parity][slice] (r, S, A, P)
  __shared__ __align__(8) uint64_t rec_bar[2];
  __shared__ __align__(8) uint64_t load_bar[2];
  __shared__ Sums wsum[kMaxWarps];
  __shared__ int32_t slot_id[kDistillMaxK];
  __shared__ float slot_p[kDistillMaxK];
  __shared__ float teacher_p, teacher_c;   // P and C
  __shared__ int teacher_bad;

  const int rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t cluster = blockIdx.x / static_cast<unsigned>(slices);
  const int64_t clusters = gridDim.x / static_cast<unsigned>(slices);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
  const float sl = a.scale * kLog2e, tau = 8.0f / sl;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&rec_bar[i], 1);
      mbar_init(&load_bar[i], 1);
    }
    fence_mbarrier_init();
  }
  __syncthreads();
  if (slices > 1) cluster_sync_all();   // every barrier exists before a peer signals it

  auto issue = [&](int b, int64_t t) {   // one thread: this block's slice of row t
    const RowShape<IT> shape(t * a.v, a.v);
    const int u0 = min(rank * per, shape.units), u1 = min(u0 + per, shape.units);
    const uint32_t bytes = static_cast<uint32_t>(u1 - u0) * 16u;
    mbar_arrive_expect_tx(&load_bar[b], bytes);
    const char* src = static_cast<const char*>(a.logits) +
                      (t * a.v + shape.head) * static_cast<int64_t>(sizeof(IT)) +
                      static_cast<int64_t>(u0) * 16;
    uint8_t* dst = buffers + b * buf_stride;
    for (uint32_t off = 0; off < bytes; off += 16384u)
      bulk_load(dst + off, src + off, min(bytes - off, 16384u), &load_bar[b]);
  };
  if (tid == 0)
    for (int b = 0; b < nbuf; ++b)
      if (cluster + b * clusters < a.T) issue(b, cluster + b * clusters);

  // the last warp's teacher slots of the next row, slot lane + 32·i in place i
  const bool teacher_warp = warp == warps - 1;
  int32_t next_id[kSlots];
  float next_t[kSlots];
  float w = 1.0f;
  auto fetch_slots = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int k = lane + 32 * i;
      next_id[i] = -1;
      next_t[i] = -CUDART_INF_F;
      if (k < a.K) {
        next_id[i] = a.ids[t * a.K + k];
        next_t[i] = a.teacher[t * a.K + k];
      }
    }
  };
  if (teacher_warp && cluster < a.T) fetch_slots(cluster);

  int k = 0;
  for (int64_t t = cluster; t < a.T; t += clusters, ++k) {
    const int par = k & 1;
    const int buf = nbuf == 2 ? par : 0;
    const uint32_t load_phase = static_cast<uint32_t>(nbuf == 2 ? k >> 1 : k) & 1u;
    const RowShape<IT> shape(t * a.v, a.v);
    const IT* row = static_cast<const IT*>(a.logits) + t * a.v;
    const int u0 = min(rank * per, shape.units), u1 = min(u0 + per, shape.units);
    const int n = u1 - u0;
    const uint4* slice = reinterpret_cast<const uint4*>(buffers + buf * buf_stride);
    w = a.weight ? a.weight[t] : 1.0f;
    if (tid == 0 && slices > 1)
      mbar_arrive_expect_tx(&rec_bar[par], static_cast<uint32_t>(slices) * 16u);
    // rank 0's edges: thread i < head element i, threads from 32 the tail
    const bool is_head = rank == 0 && tid < shape.head;
    const bool is_tail = rank == 0 && tid >= 32 && tid < 32 + shape.tail;
    const int64_t edge_j = is_head ? tid : shape.head + static_cast<int64_t>(shape.units) * kN + tid - 32;
    const float edge_x = is_head || is_tail ? to_f32(row[edge_j]) : 0.0f;

    if (teacher_warp) {
      float lp[kSlots];
      bool bad = false;
      float top = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const bool out = next_id[i] < -1 || next_id[i] >= a.v;
        bad |= out;
        if (out || next_id[i] == -1) {   // the value of an empty slot is not looked at
          next_id[i] = -1;
          next_t[i] = -CUDART_INF_F;
        }
        lp[i] = next_t[i];
        top = fmaxf(top, lp[i]);
      }
      if (a.renormalize) {
        top = warp_max(top);
        if (top == -CUDART_INF_F) top = 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          lp[i] -= top;
          if (lane + 32 * i < a.K) sum += expf(lp[i]);
        }
        sum = warp_sum(sum);
        const float log_sum = sum == 0.0f ? 0.0f : logf(sum);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) lp[i] -= log_sum;
      }
      float P = 0.0f, C = 0.0f;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (lane + 32 * i >= a.K) continue;
        const float p = next_id[i] == -1 ? 0.0f : expf(lp[i]);
        P += p;
        if (p != 0.0f) C = fmaf(p, lp[i], C);
        slot_id[lane + 32 * i] = next_id[i];
        slot_p[lane + 32 * i] = p;
      }
      P = warp_sum(P);
      C = warp_sum(C);
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) {
        teacher_p = P;
        teacher_c = C;
        teacher_bad = bad;
      }
      __syncwarp();
    }

    if (!mbar_wait_cluster_bounded(&load_bar[buf], load_phase, wait_ns)) {
      if (tid == 0 && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_TIMEOUT);
    }
    RowSums sums;
    {
      int u = tid;
      for (; u + threads < n; u += 2 * threads) {
        float x[2 * kN];
        Unit<IT>::unpack(slice[u], x);
        Unit<IT>::unpack(slice[u + threads], x + kN);
        sums.add<2 * kN, false>(x, sl, tau);
      }
      if (u < n) {
        float x[kN];
        Unit<IT>::unpack(slice[u], x);
        sums.add<kN, false>(x, sl, tau);
      }
    }
    if (is_head || is_tail) sums.add1<false>(edge_x, sl, tau);
    const Sums ws = warp_sums(sums, sl);
    if (lane == 0) wsum[warp] = ws;
    __syncthreads();
    Sums all = join_sums(warps, sl, [&](int i) { return wsum[i]; });

    // the element of the row this block holds at j, or not its own
    auto mine = [&](int j) {
      return (j >= shape.head + u0 * kN && j < shape.head + u1 * kN) ||
             (rank == 0 && (j < shape.head || j >= shape.head + shape.units * kN));
    };
    auto value = [&](int j) {
      const int q = j - shape.head - u0 * kN;
      if (q >= 0 && q < n * kN) return to_f32(reinterpret_cast<const IT*>(slice)[q]);
      return to_f32(row[j]);   // an edge, not yet written over
    };
    if (teacher_warp) {
      // fetch the next row's slots behind this row's sums
      const float r = all.m == -CUDART_INF_F ? 0.0f : all.m;
      float A = 0.0f, P = 0.0f;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int s = lane + 32 * i;
        if (s >= a.K) continue;
        const int id = slot_id[s];
        const float p = slot_p[s];
        if (id >= 0 && p != 0.0f && mine(id)) {
          A = fmaf(p, value(id) - r, A);
          P += p;
        }
      }
      A = warp_sum(A);
      P = warp_sum(P);
      if (slices > 1) {
        if (lane < slices)
          st_async_v4(mapa_shared(&rec[par][rank][0], static_cast<uint32_t>(lane)),
                      mapa_shared(&rec_bar[par], static_cast<uint32_t>(lane)), all.m, all.s, A, P);
      } else if (lane == 0) {
        rec[par][0][2] = A;
      }
      if (t + clusters < a.T) fetch_slots(t + clusters);
    }
    float A = 0.0f;
    if (slices > 1) {
      if (!mbar_wait_cluster_bounded(&rec_bar[par], static_cast<uint32_t>(k >> 1) & 1u, wait_ns)) {
        if (tid == 0 && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_TIMEOUT);
      }
      all = join_sums(slices, sl,
                      [&](int i) { return Sums{rec[par][i][0], rec[par][i][1], 0.0f}; });
    }
    const float ref = all.m == -CUDART_INF_F ? 0.0f : all.m;
    const float P = teacher_p;
    const bool any_bad = teacher_bad != 0;
    const bool dead = w == 0.0f || (P == 0.0f && !any_bad);
    const bool invalid = !dead && any_bad;
    if (rank == 0 && teacher_warp) {
      if (slices > 1) {
        // Σ_i A_i + (r_i − r)·P_i, the slices' sums moved to the common reference
        for (int i = 0; i < slices; ++i) {
          const float pi = rec[par][i][3];
          if (pi != 0.0f) {
            const float ri = rec[par][i][0];
            A += fmaf((ri == -CUDART_INF_F ? 0.0f : ri) - ref, pi, rec[par][i][2]);
          }
        }
      } else {
        __syncwarp();
        A = rec[par][0][2];
      }
      if (lane == 0) {
        const float log_s = logf(all.s);
        const float loss = fmaf(P, log_s, fmaf(-a.scale, A, teacher_c));
        a.loss[t] = dead ? 0.0f : invalid ? CUDART_NAN_F : w * loss;
        if (a.lse) a.lse[t] = fmaf(a.scale, ref, log_s);
        if (invalid && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
      }
    }

    const float c = a.grad_scale * w * a.scale;
    const float inv = 1.0f / all.s;
    const float coef = invalid ? CUDART_NAN_F : c * (P * inv);
    GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
    // the listed tokens of this block's own elements: P·q less every slot
    // that names the token, written by the first such slot
    float patch[2];
    int patch_j[2] = {-1, -1};
    if (a.dlogits != nullptr) {
      const float2 nr = make_float2(-ref, -ref), sl2 = make_float2(sl, sl);
      const float2 c2 = make_float2(coef, coef);
      GT* dst = out + shape.head + static_cast<int64_t>(u0) * kN;
      for (int u = tid; u < n; u += threads) {
        float x[kN];
        Unit<IT>::unpack(slice[u], x);
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
          const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[i], x[i + 1]), nr), sl2);
          const float2 g = __fmul2_rn(make_float2(ex2_approx(y.x), ex2_approx(y.y)), c2);
          x[i] = dead ? 0.0f : g.x;
          x[i + 1] = dead ? 0.0f : g.y;
        }
        put_unit<kN>(dst + static_cast<int64_t>(u) * kN, x);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int s = tid + h * threads;
        if (dead || s >= a.K) continue;
        const int id = slot_id[s];
        if (id < 0 || !mine(id)) continue;
        float sum = 0.0f;
        bool first = true;
        for (int q = 0; q < a.K; ++q)
          if (slot_id[q] == id) {
            if (q < s) first = false;
            sum += slot_p[q];
          }
        if (first) {
          patch_j[h] = id;
          patch[h] = invalid ? CUDART_NAN_F
                             : c * (P * (ex2_approx((value(id) - ref) * sl) * inv) - sum);
        }
      }
    }
    // every read of this row's slice, edges and slots by this block is done,
    // and its writes of P·q are ordered before the listed tokens'
    __syncthreads();
    if (a.dlogits != nullptr) {
      if (is_head || is_tail)
        put(out + edge_j, dead ? 0.0f : coef * ex2_approx((edge_x - ref) * sl));
    }
    if (tid == 0 && t + nbuf * clusters < a.T) {
      fence_proxy_async_smem();
      issue(buf, t + nbuf * clusters);
    }
    if (a.dlogits != nullptr) {
      if (shape.head + shape.tail > 0 && rank == 0) __syncthreads();   // the edges too
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (patch_j[h] >= 0) put(out + patch_j[h], patch[h]);
    }
  }
  if (slices > 1) cluster_sync_all();   // every peer's record into this block has landed
}

template <typename IT, typename GT>
tp_status distill_launch_t(const DistillArgs& a, cudaStream_t stream) {
  constexpr int64_t kN = Unit<IT>::kN;
  const int64_t units = (a.v + kN - 1) / kN;
  // Slices of a row: enough that one is at most 26 KB, so that several blocks
  // share an SM and one's writes run beside another's reads; with few rows,
  // more of them while each keeps 4 KB.
  int slices = 1;
  while (slices < kMaxSlices &&
         (units * 16 > 26 * 1024 * slices ||
          (a.T * slices * 2 <= num_sms() && units * 16 >= 8192 * slices)))
    slices *= 2;
  const int per = static_cast<int>((units + slices - 1) / slices);
  const int64_t stride = (static_cast<int64_t>(per) * 16 + 127) & ~int64_t{127};
  if (stride > kDistillMaxSlice) return TP_ERR_UNSUPPORTED;
  const int nbuf = 2 * stride <= kDistillMaxSlice ? 2 : 1;
  const int threads = stride <= 32 * 1024 ? 128 : stride <= 56 * 1024 ? 256 : 512;
  const int smem = static_cast<int>(stride * nbuf);
  int dev = 0;
  cudaGetDevice(&dev);
  static bool configured[64] = {false};
  if (!configured[dev & 63]) {
    if (cudaFuncSetAttribute(distill_kernel<IT, GT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kDistillMaxSlice)) != cudaSuccess ||
        cudaFuncSetAttribute(distill_kernel<IT, GT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return TP_ERR_CUDA;
    configured[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // clusters that can be resident at once, by launch shape
  struct Shape {
    int dev = -1, slices = 0, smem = 0, threads = 0, clusters = 0;
  };
  static thread_local Shape last;
  if (last.dev != dev || last.slices != slices || last.smem != smem || last.threads != threads) {
    int n = 0;
    cfg.gridDim = dim3(static_cast<unsigned>(slices * num_sms()));
    if (cudaOccupancyMaxActiveClusters(&n, distill_kernel<IT, GT>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = num_sms() / slices;
    }
    last.dev = dev;
    last.slices = slices;
    last.smem = smem;
    last.threads = threads;
    last.clusters = n;
  }
  const int64_t clusters = a.T < last.clusters ? a.T : last.clusters;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * slices));
  if (cudaLaunchKernelEx(&cfg, distill_kernel<IT, GT>, a, slices, per, nbuf,
                         static_cast<uint32_t>(stride), wait_limit_ns()) != cudaSuccess) {
    cudaGetLastError();
    return TP_ERR_CUDA;
  }
  note_launches(1);
  return TP_OK;
}

}  // namespace

tp_status distill_launch(const DistillArgs& a, tp_dtype dt, tp_dtype grad_dt, float* loss_sum,
                         cudaStream_t stream) {
  tp_status st;
  if (dt == TP_DTYPE_BF16)
    st = a.dlogits && grad_dt == TP_DTYPE_F32 ? distill_launch_t<__nv_bfloat16, float>(a, stream)
                                              : distill_launch_t<__nv_bfloat16, __nv_bfloat16>(a, stream);
  else
    st = a.dlogits && grad_dt == TP_DTYPE_F32 ? distill_launch_t<float, float>(a, stream)
                                              : distill_launch_t<float, __nv_bfloat16>(a, stream);
  if (st) return st;
  return loss_sum ? loss_sum_launch(a.loss, a.T, loss_sum, stream) : TP_OK;
}

}  // namespace tpl
