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
constexpr int kSeenWords = 1024;            // 32768 bits to notice a token listed twice
constexpr int kChunkUnits = 2048;           // 32 KB of a slice, the grain of its refill
constexpr int kMaxChunks = static_cast<int>((kDistillMaxSlice + 16 * kChunkUnits - 1) / (16 * kChunkUnits));

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

// 4 bytes global -> shared, waited for by the same thread.
__device__ __forceinline__ void copy_word(void* smem_dst, const void* gsrc) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem_dst)), "l"(gsrc)
               : "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
// token, p the token's summed probability.
struct SlotLists {
  int32_t* id[2];
  float* p[2];
  float* x;        // the tokens' logits, of the row at hand
  int32_t* raw_id; // all slots of the next row
  float* raw_t;
  uint32_t* seen;  // [kSeenWords], zero between rows
};

// Persistent clusters of `slices` blocks; cluster c handles rows c, c + C, …
// Block r of a cluster owns units [r·per, (r+1)·per) of each row, block 0 also
// the row's edges.  The slice lies in shared memory in chunks; a chunk is
// refilled with the next row's as soon as its gradient is written, so reads
// of one row run beside the writes of the one before.  Of a block's warps the
// last issues the copies, the one before looks after the teacher, the others
// stream.  Per row:
//   1. every streaming thread adds up its units as the chunks arrive;  barrier
//   2. the teacher warp adds A and P of the block's own tokens and sends
//      (r, S, A, P) to every block of the cluster, one 16-byte asynchronous
//      store counted on the receiver's barrier; then it turns the next row's
//      slots (loaded a row ahead) into probabilities;
//   3. the blocks combine the records in slice order and the streaming
//      threads write P·q over their slice, handing back chunk by chunk;
//   4. the teacher warp, behind a barrier, writes the listed tokens over that.
template <typename IT, typename GT>
__global__ void __launch_bounds__(kMaxThreads + 64, 2)
    distill_kernel(const DistillArgs a, int slices, int per, uint32_t buf_bytes, uint64_t wait_ns) {
  constexpr int kN = Unit<IT>::kN;
  extern __shared__ __align__(128) uint8_t buffer[];      // the slice, then the slot lists
  __shared__ __align__(16) float rec[2][kMaxSlices][4];   // [row parity][slice] (r, S, A, P)
  __shared__ __align__(8) uint64_t rec_bar[2];
  __shared__ __align__(8) uint64_t full[kMaxChunks];      // a chunk of the row has landed
  __shared__ __align__(8) uint64_t empty[kMaxChunks];     // ... and nothing reads it any more
  __shared__ Sums wsum[2][kMaxWarps];
  __shared__ float edge[2][2][8];          // [row parity] the row's two edges (block 0)
  __shared__ float teacher_p[2], teacher_c[2];
  __shared__ int teacher_bad[2];

  const int rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t cluster = blockIdx.x / static_cast<unsigned>(slices);
  const int64_t clusters = gridDim.x / static_cast<unsigned>(slices);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x) - 64, warps = threads >> 5;
  const int chunks = (per + kChunkUnits - 1) / kChunkUnits;
  const float sl = a.scale * kLog2e, tau = 8.0f / sl;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&rec_bar[i], 1);
    for (int c = 0; c < chunks; ++c) {
      mbar_init(&full[c], 1);
      // the streaming warps and, where a gradient may overwrite the logits, the teacher's
      mbar_init(&empty[c], static_cast<uint32_t>(warps) + (a.dlogits != nullptr ? 1 : 0));
    }
    fence_mbarrier_init();
  }
  __syncthreads();
  if (slices > 1) cluster_sync_all();   // every barrier exists before a peer signals it

  const volatile int never = 0;   // no role of the block cuts another's wait short
  auto timeout = [&]() {
    if (a.dev_status) atomicOr(a.dev_status, TP_DEVERR_TIMEOUT);
  };
  // the row's softmax sums over all slices (every thread of a warp calls it)
  auto row_sums = [&](int k) {
    if (slices == 1) return join_sums(warps, wsum[k & 1][min(lane, warps - 1)], sl);
    if (!mbar_wait_cluster_bounded(&rec_bar[k & 1], static_cast<uint32_t>(k >> 1) & 1u, wait_ns))
      timeout();
    const float* q = rec[k & 1][min(lane, slices - 1)];
    return join_sums(slices, Sums{q[0], q[1], 0.0f}, sl);
  };

  if (warp == warps + 1) {
    // ----------------------------------------------------------------- copies
    if (lane == 0) {
      int k = 0;
      for (int64_t t = cluster; t < a.T; t += clusters, ++k) {
        const RowShape<IT> shape(t * a.v, a.v);
        const int u0 = min(rank * per, shape.units);
        const int n = min(u0 + per, shape.units) - u0;
        const char* src = static_cast<const char*>(a.logits) +
                          (t * a.v + shape.head) * static_cast<int64_t>(sizeof(IT)) +
                          static_cast<int64_t>(u0) * 16;
        for (int c = 0; c < chunks; ++c) {
          if (k > 0 && !mbar_wait_bounded(&empty[c], static_cast<uint32_t>(k - 1) & 1u, wait_ns, &never))
            timeout();
          const int units = min(max(n - c * kChunkUnits, 0), kChunkUnits);
          mbar_arrive_expect_tx(&full[c], static_cast<uint32_t>(units) * 16u);
          if (units > 0)
            bulk_load(buffer + c * kChunkUnits * 16, src + static_cast<int64_t>(c) * kChunkUnits * 16,
                      static_cast<uint32_t>(units) * 16u, &full[c]);
        }
      }
    }
  } else if (warp == warps) {
    // ---------------------------------------------------------------- teacher
    SlotLists list;
    {
      uint8_t* at = buffer + buf_bytes;
      const int bytes = a.K * 4;
      for (int i = 0; i < 2; ++i) {
        list.id[i] = reinterpret_cast<int32_t*>(at + 2 * i * bytes);
        list.p[i] = reinterpret_cast<float*>(at + (2 * i + 1) * bytes);
      }
      list.raw_id = reinterpret_cast<int32_t*>(at + 4 * bytes);
      list.raw_t = reinterpret_cast<float*>(at + 5 * bytes);
      list.x = reinterpret_cast<float*>(at + 6 * bytes);
      list.seen = reinterpret_cast<uint32_t*>(at + 7 * bytes);
      for (int i = lane; i < kSeenWords; i += 32) list.seen[i] = 0;
      __syncwarp();
    }
    // row t's slots on their way into the lists' raw places, lane by lane
    auto fetch = [&](int64_t t) {
      for (int s = lane; s < a.K; s += 32) {
        copy_word(&list.raw_id[s], a.ids + t * a.K + s);
        copy_word(&list.raw_t[s], a.teacher + t * a.K + s);
      }
    };
    // probabilities of row t's slots and the list of this block's own; how many
    auto prepare = [&](int64_t t, int b) -> int {
      const RowShape<IT> shape(t * a.v, a.v);
      const int own0 = shape.head + min(rank * per, shape.units) * kN;
      const int own1 = shape.head + min(rank * per + per, shape.units) * kN;
      const int body1 = shape.head + shape.units * kN;
      copy_wait();
      bool bad = false;
      float top = -CUDART_INF_F;
      for (int s = lane; s < a.K; s += 32) {
        const int id = list.raw_id[s];
        const bool out = id < -1 || id >= a.v;
        bad |= out;
        if (out || id == -1) {   // the value of an empty slot is not looked at
          list.raw_id[s] = -1;
          list.raw_t[s] = -CUDART_INF_F;
        }
        top = fmaxf(top, list.raw_t[s]);
      }
      float log_sum = 0.0f;
      if (a.renormalize) {
        top = warp_max(top);
        if (top == -CUDART_INF_F) top = 0.0f;
        float sum = 0.0f;
        for (int s = lane; s < a.K; s += 32) sum += expf(list.raw_t[s] - top);
        sum = warp_sum(sum);
        log_sum = sum == 0.0f ? 0.0f : logf(sum);
      } else {
        top = 0.0f;
      }
      float P = 0.0f, C = 0.0f;
      int n = 0;
      for (int s0 = 0; s0 < a.K; s0 += 32) {
        int id = -1;
        float lp = 0.0f, p = 0.0f;
        if (s0 + lane < a.K) {
          id = list.raw_id[s0 + lane];
          lp = (list.raw_t[s0 + lane] - top) - log_sum;
          if (id != -1) p = expf(lp);
        }
        P += p;
        if (p != 0.0f) C = fmaf(p, lp, C);
        const bool own = p != 0.0f && ((id >= own0 && id < own1) ||
                                       (rank == 0 && (id < shape.head || id >= body1)));
        const uint32_t mask = __ballot_sync(0xffffffffu, own);
        if (own) {
          const int at = n + __popc(mask & ((1u << lane) - 1u));
          list.id[b][at] = id;
          list.p[b][at] = p;
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
      // A token listed twice shows as a bit of `seen` that was set already;
      // that it is one, and not two tokens on one bit, is looked up.
      bool twice = false;
      for (int e = lane; e < n; e += 32) {
        const uint32_t bit = static_cast<uint32_t>(list.id[b][e]) & (kSeenWords * 32 - 1);
        if ((atomicOr(&list.seen[bit >> 5], 1u << (bit & 31)) >> (bit & 31)) & 1u)
          for (int q = 0; q < n; ++q) twice |= q != e && list.id[b][q] == list.id[b][e];
      }
      __syncwarp();
      for (int e = lane; e < n; e += 32)
        list.seen[(static_cast<uint32_t>(list.id[b][e]) & (kSeenWords * 32 - 1)) >> 5] = 0;
      if (__any_sync(0xffffffffu, twice)) {   // one entry per token, summed in slot order
        for (int e = lane; e < n; e += 32) {
          const int id = list.id[b][e];
          float sum = 0.0f;
          bool first = true;
          for (int q = 0; q < n; ++q)
            if (list.id[b][q] == id) {
              if (q < e) first = false;
              sum += list.p[b][q];
            }
          list.raw_id[e] = first ? id : -1;
          list.raw_t[e] = sum;
        }
        __syncwarp();
        for (int e = lane; e < n; e += 32) {
          list.id[b][e] = list.raw_id[e];
          list.p[b][e] = list.raw_t[e];
        }
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
      const int par = k & 1;
      const RowShape<IT> shape(t * a.v, a.v);
      const int own0 = shape.head + min(rank * per, shape.units) * kN;
      const int own1 = shape.head + min(rank * per + per, shape.units) * kN;
      const IT* slice = reinterpret_cast<const IT*>(buffer);
      auto value = [&](int j) {
        if (a.dlogits == nullptr) return to_f32(static_cast<const IT*>(a.logits)[t * a.v + j]);
        if (j >= own0 && j < own1) return to_f32(slice[j - own0]);
        return j < shape.head ? edge[par][0][j] : edge[par][1][j - shape.head - shape.units * kN];
      };
      const float w = a.weight ? a.weight[t] : 1.0f;
      named_barrier_sync(1, static_cast<uint32_t>(threads) + 32);   // the block's sums and edges
      if (a.dlogits != nullptr)
        for (int c = 0; c < chunks; ++c)   // landed: the streaming warps have waited for them
          if (!mbar_wait_bounded(&full[c], static_cast<uint32_t>(k) & 1u, wait_ns, &never)) timeout();
      const Sums own = join_sums(warps, wsum[par][min(lane, warps - 1)], sl);
      const float own_ref = own.m == -CUDART_INF_F ? 0.0f : own.m;
      float A = 0.0f, Pown = 0.0f;
      for (int e = lane; e < n; e += 32) {
        const int id = list.id[par][e];
        if (id >= 0) {
          const float x = value(id);
          list.x[e] = x;
          A = fmaf(list.p[par][e], x - own_ref, A);
          Pown += list.p[par][e];
        }
      }
      A = warp_sum(A);
      Pown = warp_sum(Pown);
      if (slices > 1 && lane < slices)
        st_async_v4(mapa_shared(&rec[par][rank][0], static_cast<uint32_t>(lane)),
                    mapa_shared(&rec_bar[par], static_cast<uint32_t>(lane)), own.m, own.s, A, Pown);
      if (a.dlogits != nullptr && lane < chunks) mbar_arrive(&empty[lane]);   // behind the shuffles: every lane has read
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
      if (a.dlogits != nullptr) {
        named_barrier_sync(2, static_cast<uint32_t>(threads) + 32);   // P·q is written
        if (!dead) {
          const float c = any_bad ? CUDART_NAN_F : a.grad_scale * w * a.scale;
          const float inv = 1.0f / all.s;
          GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
          for (int e = lane; e < n; e += 32) {
            const int id = list.id[par][e];
            if (id >= 0)
              put(out + id, c * (P * (ex2_approx((list.x[e] - ref) * sl) * inv) - list.p[par][e]));
          }
        }
      }
      n = n_next;
    }
  } else {
    // -------------------------------------------------------------- streaming
    const uint4* slice = reinterpret_cast<const uint4*>(buffer);
    auto release = [&](int c) {   // this warp has read chunk c for the last time
      __syncwarp();
      if (lane == 0) {
        fence_proxy_async_smem();   // the reads come before the refill's writes
        mbar_arrive(&empty[c]);
      }
    };
    constexpr int kBatch = 16 / kN;   // units a thread has in hand: 16 logits
    constexpr uint32_t kInf = Unit<IT>::kMinusInf;
    const uint4 fill = make_uint4(kInf, kInf, kInf, kInf);
    int k = 0;
    for (int64_t t = cluster; t < a.T; t += clusters, ++k) {
      const int par = k & 1;
      const RowShape<IT> shape(t * a.v, a.v);
      const int u0 = min(rank * per, shape.units);
      const int n = min(u0 + per, shape.units) - u0;
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
        edge[par][is_head ? 0 : 1][is_head ? tid : tid - 32] = edge_x;
      }
      RowSums sums;
      for (int c = 0; c < chunks; ++c) {
        if (!mbar_wait_bounded(&full[c], static_cast<uint32_t>(k) & 1u, wait_ns, &never)) timeout();
        const int end = min((c + 1) * kChunkUnits, n);
        for (int u = c * kChunkUnits + tid; u < end; u += kBatch * threads) {
          float x[kBatch * kN];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            Unit<IT>::unpack(u + i * threads < end ? slice[u + i * threads] : fill, x + i * kN);
          sums.add<kBatch * kN, false>(x, sl, tau);
        }
        if (a.dlogits == nullptr) release(c);
      }
      if (is_head || is_tail) sums.add1<false>(edge_x, sl, tau);
      const Sums ws = warp_sums(sums, sl);
      if (lane == 0) wsum[par][warp] = ws;
      named_barrier_sync(1, static_cast<uint32_t>(threads) + 32);
      if (a.dlogits == nullptr) {
        if (slices > 1) row_sums(k);   // the records of row k+2 reuse this row's places
        continue;
      }
      const Sums all = row_sums(k);
      const float ref = all.m == -CUDART_INF_F ? 0.0f : all.m;
      const float P = teacher_p[par];
      const bool any_bad = teacher_bad[par] != 0;
      const bool dead = w == 0.0f || (P == 0.0f && !any_bad);
      const float coef = any_bad ? CUDART_NAN_F : a.grad_scale * w * a.scale * (P * (1.0f / all.s));
      GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
      GT* dst = out + shape.head + static_cast<int64_t>(u0) * kN;
      const float2 nr = make_float2(-ref, -ref), sl2 = make_float2(sl, sl);
      const float2 c2 = make_float2(coef, coef);
      for (int c = 0; c < chunks; ++c) {
        const int end = min((c + 1) * kChunkUnits, n);
        if (dead) {
          const float z[kN] = {};
          for (int u = c * kChunkUnits + tid; u < end; u += threads)
            put_unit<kN>(dst + static_cast<int64_t>(u) * kN, z);
        } else {
          for (int u = c * kChunkUnits + tid; u < end; u += kBatch * threads) {
            uint4 w4[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              w4[i] = u + i * threads < end ? slice[u + i * threads] : fill;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              float x[kN];
              Unit<IT>::unpack(w4[i], x);
#pragma unroll
              for (int q = 0; q < kN; q += 2) {
                const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[q], x[q + 1]), nr), sl2);
                const float2 g = __fmul2_rn(make_float2(ex2_approx(y.x), ex2_approx(y.y)), c2);
                x[q] = g.x;
                x[q + 1] = g.y;
              }
              if (u + i * threads < end)
                put_unit<kN>(dst + static_cast<int64_t>(u + i * threads) * kN, x);
            }
          }
        }
        release(c);
      }
      if (is_head || is_tail)
        put(out + edge_j, dead ? 0.0f : coef * ex2_approx((edge_x - ref) * sl));
      // the teacher warp's writes come after these; nothing here waits
      named_barrier_arrive(2, static_cast<uint32_t>(threads) + 32);
    }
  }
  __syncthreads();
  if (slices > 1) cluster_sync_all();   // every peer's record into this block has landed
}

template <typename IT, typename GT>
tp_status distill_launch_t(const DistillArgs& a, cudaStream_t stream) {
  constexpr int64_t kN = Unit<IT>::kN;
  const int64_t units = (a.v + kN - 1) / kN;
  // Slices of a row: at most 108 KB, so that two blocks share an SM and one's
  // barriers and exchanges run beside the other's sweeps; with few rows, more
  // of them while each keeps 4 KB.
  int slices = 1;
  while (slices < kMaxSlices &&
         (units * 16 > 108 * 1024 * slices ||
          (a.T * slices * 2 <= num_sms() && units * 16 >= 8192 * slices)))
    slices *= 2;
  if (const char* e = getenv("TPX_SL")) slices = atoi(e);
  const int per = static_cast<int>((units + slices - 1) / slices);
  const int64_t slice = (static_cast<int64_t>(per) * 16 + 127) & ~int64_t{127};
  if (slice > kDistillMaxSlice) return TP_ERR_UNSUPPORTED;
  int threads = slice <= 16 * 1024 ? 128 : slice <= 50 * 1024 ? 256 : 512;
  if (const char* e = getenv("TPX_NT")) threads = atoi(e);
  const int smem = static_cast<int>(slice + 28 * a.K + 4 * kSeenWords);   // and the slot lists
  int dev = 0;
  cudaGetDevice(&dev);
  static bool configured[64] = {false};
  if (!configured[dev & 63]) {
    if (cudaFuncSetAttribute(distill_kernel<IT, GT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kDistillMaxSlice + 28 * kDistillMaxK +
                                              4 * kSeenWords)) != cudaSuccess ||
        cudaFuncSetAttribute(distill_kernel<IT, GT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return TP_ERR_CUDA;
    configured[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(static_cast<unsigned>(threads + 64));
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
  if (cudaLaunchKernelEx(&cfg, distill_kernel<IT, GT>, a, slices, per,
                         static_cast<uint32_t>(slice), wait_limit_ns()) != cudaSuccess) {
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
