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
#include <cstdlib>

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

// A block's list of the listed tokens that lie in its slice, one for the row
// at hand and one for the next: id −1 where an earlier entry names the same
// token, p the token's summed probability (later the gradient written there).
struct SlotLists {
  int32_t* id[2];
  float* p[2];
  int32_t* raw_id;
  float* raw_p;
};

// Persistent clusters of `slices` blocks; cluster c handles rows c, c + C, …
// Block r of a cluster owns units [r·per, (r+1)·per) of each row, staged by
// bulk copies `nbuf` rows ahead, block 0 also the row's edges.  The last warp
// of a block looks after the teacher, the others stream.  Per row:
//   1. every streaming thread adds up its units;  block barrier
//   2. the teacher warp adds A and P of the block's own tokens and sends
//      (r, S, A, P) to every block of the cluster, one 16-byte asynchronous
//      store counted on the receiver's barrier; then it turns the next row's
//      slots (loaded a row ahead) into probabilities;
//   3. the blocks combine the records in slice order and the streaming
//      threads write P·q over their slice;  block barrier
//   4. the teacher warp writes the listed tokens over that, and the buffer is
//      refilled.
template <typename IT, typename GT>
__global__ void __launch_bounds__(kMaxThreads + 32, 1)
    distill_kernel(const DistillArgs a, int slices, int per, int nbuf, uint32_t buf_stride,
                   uint64_t wait_ns) {
  constexpr int kN = Unit<IT>::kN;
  extern __shared__ __align__(128) uint8_t buffers[];     // the slices, then the slot lists
  __shared__ __align__(16) float rec[2][kMaxSlices][4];   // [row parity][slice] (r, S, A, P)
  __shared__ __align__(8) uint64_t rec_bar[2];
  __shared__ __align__(8) uint64_t load_bar[2];
  __shared__ Sums wsum[kMaxWarps];
  __shared__ float edge[2][8];             // the row's edges (block 0)
  __shared__ float teacher_p[2], teacher_c[2];
  __shared__ int teacher_bad[2];

  const int rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t cluster = blockIdx.x / static_cast<unsigned>(slices);
  const int64_t clusters = gridDim.x / static_cast<unsigned>(slices);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x) - 32, warps = threads >> 5;
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

  auto timeout = [&]() {
    if (a.dev_status) atomicOr(a.dev_status, TP_DEVERR_TIMEOUT);
  };
  // the row's softmax sums over all slices (every thread of a warp calls it)
  auto row_sums = [&](int k) {
    if (slices == 1) return join_sums(warps, wsum[min(lane, warps - 1)], sl);
    if (!mbar_wait_cluster_bounded(&rec_bar[k & 1], static_cast<uint32_t>(k >> 1) & 1u, wait_ns))
      timeout();
    const float* q = rec[k & 1][min(lane, slices - 1)];
    return join_sums(slices, Sums{q[0], q[1], 0.0f}, sl);
  };

  if (warp == warps) {
    // ---------------------------------------------------------------- teacher
    SlotLists list;
    {
      uint8_t* at = buffers + nbuf * buf_stride;
      const int bytes = a.K * 4;
      for (int i = 0; i < 2; ++i) {
        list.id[i] = reinterpret_cast<int32_t*>(at + 2 * i * bytes);
        list.p[i] = reinterpret_cast<float*>(at + (2 * i + 1) * bytes);
      }
      list.raw_id = reinterpret_cast<int32_t*>(at + 4 * bytes);
      list.raw_p = reinterpret_cast<float*>(at + 5 * bytes);
    }
    int32_t next_id[kSlots];   // slot lane + 32·i of the row after the prepared one
    float next_t[kSlots];
    auto fetch = [&](int64_t t) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int s = lane + 32 * i;
        next_id[i] = -1;
        next_t[i] = -CUDART_INF_F;
        if (s < a.K) {
          next_id[i] = a.ids[t * a.K + s];
          next_t[i] = a.teacher[t * a.K + s];
        }
      }
    };
    // probabilities of row t's slots and the list of this block's own; how many
    auto prepare = [&](int64_t t, int b) -> int {
      const RowShape<IT> shape(t * a.v, a.v);
      const int own0 = shape.head + min(rank * per, shape.units) * kN;
      const int own1 = shape.head + min(rank * per + per, shape.units) * kN;
      const int body1 = shape.head + shape.units * kN;
      bool bad = false;
      float top = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (32 * i >= a.K) break;
        const bool out = next_id[i] < -1 || next_id[i] >= a.v;
        bad |= out;
        if (out || next_id[i] == -1) {   // the value of an empty slot is not looked at
          next_id[i] = -1;
          next_t[i] = -CUDART_INF_F;
        }
        top = fmaxf(top, next_t[i]);
      }
      if (a.renormalize) {
        top = warp_max(top);
        if (top == -CUDART_INF_F) top = 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          if (32 * i >= a.K) break;
          next_t[i] -= top;
          sum += expf(next_t[i]);
        }
        sum = warp_sum(sum);
        const float log_sum = sum == 0.0f ? 0.0f : logf(sum);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          if (32 * i >= a.K) break;
          next_t[i] -= log_sum;
        }
      }
      float P = 0.0f, C = 0.0f;
      int n = 0;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (32 * i >= a.K) break;
        const int id = next_id[i];
        const float p = id == -1 ? 0.0f : expf(next_t[i]);
        P += p;
        if (p != 0.0f) C = fmaf(p, next_t[i], C);
        const bool own = p != 0.0f && ((id >= own0 && id < own1) ||
                                       (rank == 0 && (id < shape.head || id >= body1)));
        const uint32_t mask = __ballot_sync(0xffffffffu, own);
        if (own) {
          const int at = n + __popc(mask & ((1u << lane) - 1u));
          list.raw_id[at] = id;
          list.raw_p[at] = p;
        }
        n += __popc(mask);
      }
      P = warp_sum(P);
      C = warp_sum(C);
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) {
        teacher_p[b] = P;
        teacher_c[b] = C;
        teacher_bad[b] = bad;
      }
      __syncwarp();
      for (int e = lane; e < n; e += 32) {   // one entry per token, summed in slot order
        const int id = list.raw_id[e];
        float sum = 0.0f;
        bool first = true;
        for (int q = 0; q < n; ++q)
          if (list.raw_id[q] == id) {
            if (q < e) first = false;
            sum += list.raw_p[q];
          }
        list.id[b][e] = first ? id : -1;
        list.p[b][e] = sum;
      }
      __syncwarp();
      return n;
    };

    int n = 0;
    if (cluster < a.T) {
      fetch(cluster);
      n = prepare(cluster, 0);
      if (cluster + clusters < a.T) fetch(cluster + clusters);
    }
    int k = 0;
    for (int64_t t = cluster; t < a.T; t += clusters, ++k) {
      const int par = k & 1, buf = nbuf == 2 ? par : 0;
      const RowShape<IT> shape(t * a.v, a.v);
      const int own0 = shape.head + min(rank * per, shape.units) * kN;
      const int own1 = shape.head + min(rank * per + per, shape.units) * kN;
      const IT* slice = reinterpret_cast<const IT*>(buffers + buf * buf_stride);
      auto value = [&](int j) {
        if (j >= own0 && j < own1) return to_f32(slice[j - own0]);
        return j < shape.head ? edge[0][j] : edge[1][j - shape.head - shape.units * kN];
      };
      const float w = a.weight ? a.weight[t] : 1.0f;
      __syncthreads();                          // the block's sums and edges
      if (!mbar_wait_cluster_bounded(&load_bar[buf],
                                     static_cast<uint32_t>(nbuf == 2 ? k >> 1 : k) & 1u, wait_ns))
        timeout();
      const Sums own = join_sums(warps, wsum[min(lane, warps - 1)], sl);
      const float own_ref = own.m == -CUDART_INF_F ? 0.0f : own.m;
      float A = 0.0f, Pown = 0.0f;
      for (int e = lane; e < n; e += 32) {
        const int id = list.id[par][e];
        if (id >= 0) {
          A = fmaf(list.p[par][e], value(id) - own_ref, A);
          Pown += list.p[par][e];
        }
      }
      A = warp_sum(A);
      Pown = warp_sum(Pown);
      if (slices > 1 && lane < slices)
        st_async_v4(mapa_shared(&rec[par][rank][0], static_cast<uint32_t>(lane)),
                    mapa_shared(&rec_bar[par], static_cast<uint32_t>(lane)), own.m, own.s, A, Pown);
      int n_next = 0;
      if (t + clusters < a.T) {
        n_next = prepare(t + clusters, par ^ 1);
        if (t + 2 * clusters < a.T) fetch(t + 2 * clusters);
      }
      const Sums all = row_sums(k);
      const float ref = all.m == -CUDART_INF_F ? 0.0f : all.m;
      const float P = teacher_p[par];
      const bool any_bad = teacher_bad[par] != 0;
      const bool dead = w == 0.0f || (P == 0.0f && !any_bad);
      if (rank == 0) {
        if (slices > 1) {   // the slices' A moved to the common reference, in slice order
          A = 0.0f;
          for (int i = 0; i < slices; ++i) {
            const float* q = rec[par][i];
            if (q[3] != 0.0f) A += fmaf((q[0] == -CUDART_INF_F ? 0.0f : q[0]) - ref, q[3], q[2]);
          }
        }
        if (lane == 0) {
          const float log_s = logf(all.s);
          const float loss = fmaf(P, log_s, fmaf(-a.scale, A, teacher_c[par]));
          a.loss[t] = dead ? 0.0f : any_bad ? CUDART_NAN_F : w * loss;
          if (a.lse) a.lse[t] = fmaf(a.scale, ref, log_s);
          if (!dead && any_bad && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
        }
      }
      const bool patches = a.dlogits != nullptr && !dead;
      if (patches) {
        const float c = any_bad ? CUDART_NAN_F : a.grad_scale * w * a.scale;
        const float inv = 1.0f / all.s;
        for (int e = lane; e < n; e += 32) {
          const int id = list.id[par][e];
          if (id >= 0)
            list.p[par][e] = c * (P * (ex2_approx((value(id) - ref) * sl) * inv) - list.p[par][e]);
        }
      }
      __syncthreads();                          // P·q is written, the slice has been read
      if (patches) {
        GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
        for (int e = lane; e < n; e += 32) {
          const int id = list.id[par][e];
          if (id >= 0) put(out + id, list.p[par][e]);
        }
      }
      n = n_next;
    }
  } else {
    // -------------------------------------------------------------- streaming
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
    int k = 0;
    for (int64_t t = cluster; t < a.T; t += clusters, ++k) {
      const int par = k & 1, buf = nbuf == 2 ? par : 0;
      const RowShape<IT> shape(t * a.v, a.v);
      const int u0 = min(rank * per, shape.units);
      const int n = min(u0 + per, shape.units) - u0;
      const uint4* slice = reinterpret_cast<const uint4*>(buffers + buf * buf_stride);
      const float w = a.weight ? a.weight[t] : 1.0f;
      // this row's records: one arrival here, 16 bytes from each slice
      if (tid == 0 && slices > 1)
        mbar_arrive_expect_tx(&rec_bar[par], static_cast<uint32_t>(slices) * 16u);
      const bool is_head = rank == 0 && tid < shape.head;
      const bool is_tail = rank == 0 && tid >= 32 && tid < 32 + shape.tail;
      const int64_t edge_j =
          is_head ? tid : shape.head + static_cast<int64_t>(shape.units) * kN + tid - 32;
      float edge_x = 0.0f;
      if (is_head || is_tail) {
        edge_x = to_f32(static_cast<const IT*>(a.logits)[t * a.v + edge_j]);
        edge[is_head ? 0 : 1][is_head ? tid : tid - 32] = edge_x;
      }
      if (!mbar_wait_cluster_bounded(&load_bar[buf],
                                     static_cast<uint32_t>(nbuf == 2 ? k >> 1 : k) & 1u, wait_ns))
        timeout();
      RowSums sums;
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
      if (is_head || is_tail) sums.add1<false>(edge_x, sl, tau);
      const Sums ws = warp_sums(sums, sl);
      if (lane == 0) wsum[warp] = ws;
      __syncthreads();
      const Sums all = row_sums(k);
      if (a.dlogits != nullptr) {
        const float ref = all.m == -CUDART_INF_F ? 0.0f : all.m;
        const float P = teacher_p[par];
        const bool any_bad = teacher_bad[par] != 0;
        const bool dead = w == 0.0f || (P == 0.0f && !any_bad);
        const float coef =
            any_bad ? CUDART_NAN_F : a.grad_scale * w * a.scale * (P * (1.0f / all.s));
        GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
        GT* dst = out + shape.head + static_cast<int64_t>(u0) * kN;
        if (dead) {
          const float z[kN] = {};
          for (u = tid; u < n; u += threads) put_unit<kN>(dst + static_cast<int64_t>(u) * kN, z);
        } else {
          const float2 nr = make_float2(-ref, -ref), sl2 = make_float2(sl, sl);
          const float2 c2 = make_float2(coef, coef);
#pragma unroll 2
          for (u = tid; u < n; u += threads) {
            float x[kN];
            Unit<IT>::unpack(slice[u], x);
#pragma unroll
            for (int i = 0; i < kN; i += 2) {
              const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[i], x[i + 1]), nr), sl2);
              const float2 g = __fmul2_rn(make_float2(ex2_approx(y.x), ex2_approx(y.y)), c2);
              x[i] = g.x;
              x[i + 1] = g.y;
            }
            put_unit<kN>(dst + static_cast<int64_t>(u) * kN, x);
          }
        }
        if (is_head || is_tail)
          put(out + edge_j, dead ? 0.0f : coef * ex2_approx((edge_x - ref) * sl));
      }
      // every read of this row's slice is done, and the writes of P·q are
      // ordered before the listed tokens'
      __syncthreads();
      if (tid == 0 && t + nbuf * clusters < a.T) {
        fence_proxy_async_smem();
        issue(buf, t + nbuf * clusters);
      }
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
  if (const char* e = getenv("TPX_SL")) slices = atoi(e);
  const int per = static_cast<int>((units + slices - 1) / slices);
  const int64_t stride = (static_cast<int64_t>(per) * 16 + 127) & ~int64_t{127};
  if (stride > kDistillMaxSlice) return TP_ERR_UNSUPPORTED;
  const int nbuf = 2 * stride <= kDistillMaxSlice ? 2 : 1;
  int threads = stride <= 32 * 1024 ? 128 : stride <= 56 * 1024 ? 256 : 512;
  if (const char* e = getenv("TPX_NT")) threads = atoi(e);
  const int smem = static_cast<int>(stride * nbuf + 24 * a.K);   // and the slot lists
  int dev = 0;
  cudaGetDevice(&dev);
  static bool configured[64] = {false};
  if (!configured[dev & 63]) {
    if (cudaFuncSetAttribute(distill_kernel<IT, GT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kDistillMaxSlice + 24 * kDistillMaxK)) != cudaSuccess ||
        cudaFuncSetAttribute(distill_kernel<IT, GT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return TP_ERR_CUDA;
    configured[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(static_cast<unsigned>(threads + 32));
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
