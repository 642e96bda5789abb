// distill.cu — loss of softmax(scale·logits) against a teacher's top entries,
// and its gradient, in one pass over the logits.
//
//   p_k: the teacher's probabilities on K listed tokens, P = Σ p_k,
//   C = Σ p_k·log p_k,  r = max x,  S = Σ exp(scale·(x − r)),
//   A = Σ p_k·(x_{id_k} − r)
//   loss = w·(C − scale·A + P·log S)
//   dlogits_j = grad_scale·w·scale·(P·exp(scale·(x_j − r))/S − Σ_{k: id_k = j} p_k)
//
// Every logit is needed twice, once for S and once for the gradient.  A
// cluster of up to eight blocks holds one row, each block its slice in
// registers while the next rows' slices arrive in shared memory: HBM sees each
// logit read once and each gradient written once, and the writes of one row run
// beside the reads of the next.  fp32 rows are held as the exponentials, each
// taken once; bf16 rows as they are, packed, each exponential taken twice.
// Rows of weight 0 are read like the others (lse needs them) and written as
// zeros.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "rowwise.cuh"
#include "sm100_ptx.cuh"

namespace tpl {
namespace {

constexpr int kMaxSlices = 8;

// Blocks of NT streaming threads with R units each that the registers of an
// SM are shared by.
constexpr int blocks_per_sm(int R, int NT) {
  return NT == 128 ? (R <= 4 ? 8 : 4) : NT == 256 || R <= 9 ? 2 : 1;
}
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

// 8 bytes global -> shared, waited for by the same thread.
__device__ __forceinline__ void copy_entry(int2* smem_dst, const int2* gsrc) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(smem_dst)), "l"(gsrc)
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

// ---------------------------------------------------------------------------
// the teacher's slots
// ---------------------------------------------------------------------------
// What the rows' clusters need of the teacher, worked out once per row:
// entries [T, K] of (token or −1, its probability), a token listed twice
// merged into its first slot; info [T] of (P, C, any bad id, weight).
struct Slots {
  const int2* entries;
  const float4* info;
};

constexpr int kPrepWarps = 4;

// The teacher's probabilities of one row in one warp, slot lane + 32·i in
// place i: ids with −1 for empty and bad slots and those of probability 0,
// log p and p.  The sums run over the lanes' slots and then by shuffles, the
// same order every time.
template <int S>
struct RowSlots {
  int32_t id[S];
  float lp[S], p[S];
  float P, C;    // Σ p, Σ p·log p
  bool bad;

  __device__ __forceinline__ RowSlots(const DistillArgs& a, int64_t t, int lane) {
    bad = false;
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int s = lane + 32 * i;
      id[i] = -1;
      lp[i] = -CUDART_INF_F;
      if (s < a.K) {
        id[i] = a.ids[t * a.K + s];
        lp[i] = a.teacher[t * a.K + s];
      }
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const bool out = id[i] < -1 || id[i] >= a.v;
      bad |= out;
      if (out || id[i] == -1) {   // the value of an empty slot is not looked at
        id[i] = -1;
        lp[i] = -CUDART_INF_F;
      }
      top = fmaxf(top, lp[i]);
    }
    if (a.renormalize) {
      top = warp_max(top);
      if (top == -CUDART_INF_F) top = 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        lp[i] -= top;
        sum += expf(lp[i]);
      }
      sum = warp_sum(sum);
      const float log_sum = sum == 0.0f ? 0.0f : logf(sum);
#pragma unroll
      for (int i = 0; i < S; ++i) lp[i] -= log_sum;
    }
    P = C = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      p[i] = id[i] == -1 ? 0.0f : expf(lp[i]);
      P += p[i];
      if (p[i] != 0.0f) C = fmaf(p[i], lp[i], C);
      else id[i] = -1;
    }
    P = warp_sum(P);
    C = warp_sum(C);
    bad = __any_sync(0xffffffffu, bad);
  }
};

// One warp per row; S slots per lane.
template <int S>
__global__ void __launch_bounds__(kPrepWarps * 32)
    distill_slots_kernel(const DistillArgs a, int2* __restrict__ entries,
                         float4* __restrict__ info) {
  constexpr int kSeenWords = 128 * S;   // 128 bits for every slot, to notice a token listed twice
  __shared__ __align__(16) uint32_t seen_bits[kPrepWarps][kSeenWords];   // cleared 16 bytes at a time
  __shared__ int2 listed[kPrepWarps][32 * S];
  grid_dependents_launch();   // the rows' kernel reads nothing of this one before it has ended
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kPrepWarps + warp;
  if (t >= a.T) return;
  uint32_t* seen = seen_bits[warp];
#pragma unroll
  for (int i = 0; i < S; ++i)
    reinterpret_cast<uint4*>(seen)[lane + 32 * i] = make_uint4(0, 0, 0, 0);
  RowSlots<S> r(a, t, lane);
  __syncwarp();
  uint32_t again = 0;   // bit i: another slot had the bit of slot i's token
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (r.id[i] >= 0) {
      const uint32_t bit = static_cast<uint32_t>(r.id[i]) & (kSeenWords * 32 - 1);
      again |= ((atomicOr(&seen[bit >> 5], 1u << (bit & 31)) >> (bit & 31)) & 1u) << i;
    }
  bool twice = false;   // (the whole warp's answer)
#pragma unroll
  for (int i = 0; i < S; ++i)
    // a token twice, or two tokens on one bit: its slots are counted
    for (uint32_t m = __ballot_sync(0xffffffffu, (again >> i) & 1u); m; m &= m - 1) {
      const int32_t id = __shfl_sync(0xffffffffu, r.id[i], __ffs(m) - 1);
      int n = 0;
#pragma unroll
      for (int q = 0; q < S; ++q) n += r.id[q] == id;
      twice |= __reduce_add_sync(0xffffffffu, n) > 1;
    }
  if (twice) {
#pragma unroll
    for (int i = 0; i < S; ++i)
      listed[warp][lane + 32 * i] = make_int2(r.id[i], __float_as_int(r.p[i]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float sum = 0.0f;
      bool first = true;
#pragma unroll 8
      for (int q = 0; q < 32 * S; ++q) {   // in slot order
        const int2 e = listed[warp][q];
        if (e.x == r.id[i]) {
          if (q < lane + 32 * i) first = false;
          sum += __int_as_float(e.y);
        }
      }
      r.p[i] = sum;
      if (!first) r.id[i] = -1;
    }
  }
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (lane + 32 * i < a.K)
      entries[t * a.K + lane + 32 * i] = make_int2(r.id[i], __float_as_int(r.p[i]));
  if (lane == 0)
    info[t] = make_float4(r.P, r.C, r.bad ? 1.0f : 0.0f, a.weight ? a.weight[t] : 1.0f);
}

// Without a gradient the logits are needed once: the rows' sums come from the
// log-probability kernel (sums [T] of (r, log S)), and one warp per row gathers
// the listed logits, beside that kernel's last rows.
template <typename IT, int S>
__global__ void __launch_bounds__(kPrepWarps * 32)
    distill_loss_kernel(const DistillArgs a, const float2* sums) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kPrepWarps + (threadIdx.x >> 5);
  grid_dependents_launch();
  if (t >= a.T) return;
  const RowSlots<S> r(a, t, lane);
  float x[S];
#pragma unroll
  for (int i = 0; i < S; ++i)
    x[i] = r.id[i] >= 0 ? to_f32(static_cast<const IT*>(a.logits)[t * a.v + r.id[i]]) : 0.0f;
  grid_dependency_wait();   // nothing above is written by the kernel before
  const float2 rs = sums[t];
  float A = 0.0f;
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (r.id[i] >= 0) A = fmaf(r.p[i], x[i] - rs.x, A);
  A = warp_sum(A);
  if (lane == 0) {
    const float w = a.weight ? a.weight[t] : 1.0f;
    const bool dead = w == 0.0f || (r.P == 0.0f && !r.bad);
    const float loss = fmaf(r.P, rs.y, fmaf(-a.scale, A, r.C));
    a.loss[t] = dead ? 0.0f : r.bad ? CUDART_NAN_F : w * loss;
    if (!dead && r.bad && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
  }
}

// ---------------------------------------------------------------------------
// the rows
// ---------------------------------------------------------------------------
// One thread's R units between the two uses of a row.  fp32 logits are kept
// as e = exp(scale·(x − m_w)) against the warp's maximum, one register each;
// bf16 logits stay packed, two to a register, and their exponentials are taken
// a second time: twice the rows fit the registers, and it is rows in flight
// that hide the exchange between a row's blocks.
template <typename IT, int R>
struct Held;

template <int R>
struct Held<float, R> {
  float e[R * 4];
  float m;   // the warp's maximum, 0 for −inf
  __device__ __forceinline__ void take(int i, uint4 w) { Unit<float>::unpack(w, e + 4 * i); }
  __device__ __forceinline__ float maximum(float mx) const {
#pragma unroll
    for (int i = 0; i < R * 4; i += 2) mx = max3f(mx, e[i], e[i + 1]);
    return mx;
  }
  __device__ __forceinline__ float sum(float ref, float sl) {
    m = ref;
    const float2 nr = make_float2(-ref, -ref), sl2 = make_float2(sl, sl);
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < R * 4; i += 2) {
      const float2 y = __fmul2_rn(__fadd2_rn(make_float2(e[i], e[i + 1]), nr), sl2);
      e[i] = ex2_approx(y.x);
      e[i + 1] = ex2_approx(y.y);
      s = __fadd2_rn(s, make_float2(e[i], e[i + 1]));
    }
    return s.x + s.y;
  }
  // coef·exp(scale·(x − ref)) of unit i
  __device__ __forceinline__ void gradient(int i, float ref, float sl, float coef, float* g) const {
    const float f = coef * ex2_approx((m - ref) * sl);
    const float2 f2 = make_float2(f, f);
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const float2 p = __fmul2_rn(make_float2(e[4 * i + q], e[4 * i + q + 1]), f2);
      g[q] = p.x;
      g[q + 1] = p.y;
    }
  }
};

template <int R>
struct Held<__nv_bfloat16, R> {
  uint4 w[R];
  __device__ __forceinline__ void take(int i, uint4 x) { w[i] = x; }
  __device__ __forceinline__ float maximum(float mx) const {
    __nv_bfloat162 m2 = __float2bfloat162_rn(-CUDART_INF_F);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m2 = __hmax2(m2, *reinterpret_cast<const __nv_bfloat162*>(&q[j]));
    }
    return max3f(mx, __low2float(m2), __high2float(m2));
  }
  __device__ __forceinline__ float sum(float ref, float sl) {
    const float2 nr = make_float2(-ref, -ref), sl2 = make_float2(sl, sl);
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float x[8];
      Unit<__nv_bfloat16>::unpack(w[i], x);
#pragma unroll
      for (int q = 0; q < 8; q += 2) {
        const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[q], x[q + 1]), nr), sl2);
        s = __fadd2_rn(s, make_float2(ex2_approx(y.x), ex2_approx(y.y)));
      }
    }
    return s.x + s.y;
  }
  __device__ __forceinline__ void gradient(int i, float ref, float sl, float coef, float* g) const {
    const float2 nr = make_float2(-ref, -ref), sl2 = make_float2(sl, sl);
    const float2 c2 = make_float2(coef, coef);
    uint4 q4 = w[i];   // unpacked anew, not kept in registers since the sum
    asm volatile("" : "+r"(q4.x), "+r"(q4.y), "+r"(q4.z), "+r"(q4.w));
    float x[8];
    Unit<__nv_bfloat16>::unpack(q4, x);
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
      const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x[q], x[q + 1]), nr), sl2);
      const float2 p = __fmul2_rn(make_float2(ex2_approx(y.x), ex2_approx(y.y)), c2);
      g[q] = p.x;
      g[q + 1] = p.y;
    }
  }
};

// Persistent clusters of `slices` blocks; cluster c handles rows c, c + C, …
// Block r of a cluster owns units [r·per, (r+1)·per) of each row, per <= R·NT,
// block 0 also the row's edges.  NT threads stream and one more warp looks
// after the teacher.  Per row:
//   1. the streaming threads take their R units from shared memory into
//      registers and add them up; the teacher warp picks up the logits of the
//      block's own listed tokens; barrier, and the buffer is refilled `nbuf`
//      rows ahead;
//   2. warp 0 sends the block's (r, S) to every block of the cluster, one
//      16-byte asynchronous store counted on the receiver's barrier; the
//      teacher warp sends A and P of its own tokens to block 0 the same way
//      and lists its tokens of the next row;
//   3. the blocks combine the records in slice order and the streaming
//      threads write P·q over their slice;
//   4. the teacher warp, behind a barrier, writes the listed tokens over that;
//      block 0's writes the loss.
//
// Waits are bounded, and a block of which one has run out waits no more: it
// arms no barrier again (the last phase may be incomplete), asks for no copy and
// sends no record, so its peers' waits run out in turn and the call ends a few
// limits later, whatever its rows.
template <typename IT, typename GT, int R, int NT>
__global__ void __launch_bounds__(NT + 32, blocks_per_sm(R, NT))
    distill_kernel(const DistillArgs a, const Slots slots, int slices, int per, int nbuf,
                   uint32_t buf_stride, uint64_t wait_ns, int64_t stall_row) {
  constexpr int kN = Unit<IT>::kN;
  constexpr int kWarps = NT / 32;
  extern __shared__ __align__(128) uint8_t buffers[];       // the slices, then the slot lists
  __shared__ __align__(16) float rec[2][kMaxSlices][4];     // [row parity][slice] (r, S)
  __shared__ __align__(16) float own_rec[2][kMaxSlices][4]; // [row parity][slice] (A, P, r), block 0
  __shared__ __align__(8) uint64_t rec_bar[2];
  __shared__ __align__(8) uint64_t own_bar[2];
  __shared__ __align__(8) uint64_t load_bar[2];
  __shared__ __align__(16) float wmax[2][kWarps], wsum[2][kWarps];   // [row parity] the warps' m, S
  __shared__ float4 row_info[2];                            // [row parity]
  __shared__ volatile int late;    // a wait of this block has run out
  __shared__ int asked;            // rows whose copies thread 32 has asked for

  const int rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t cluster = blockIdx.x / static_cast<unsigned>(slices);
  const int64_t clusters = gridDim.x / static_cast<unsigned>(slices);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float sl = a.scale * kLog2e;

  grid_dependents_launch();
  if (tid == 0) {
    late = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&rec_bar[i], 1);
      mbar_init(&own_bar[i], 1);
      mbar_init(&load_bar[i], 1);
    }
    fence_mbarrier_init();
  }
  __syncthreads();
  if (slices > 1) cluster_sync_all();   // every barrier exists before a peer signals it

  auto wait = [&](uint64_t* bar, int phase) {
    const uint32_t parity = static_cast<uint32_t>(phase) & 1u;
    if (mbar_test_cluster(bar, parity) || late) return;
    if (!mbar_wait_cluster_bounded(bar, parity, wait_ns, &late)) {
      late = 1;
      if (a.dev_status) atomicOr(a.dev_status, TP_DEVERR_TIMEOUT);
    }
  };
  auto wait_slice = [&](int k) {
    wait(&load_bar[nbuf == 2 ? k & 1 : 0], nbuf == 2 ? k >> 1 : k);
  };
  // this block's sums of row k, and the row's over all slices (a whole warp
  // calls it)
  auto block_sums = [&](int k) {
    if constexpr (kWarps == 4) {
      const float4 m = *reinterpret_cast<const float4*>(wmax[k & 1]);
      const float4 s = *reinterpret_cast<const float4*>(wsum[k & 1]);
      const float mx = fmaxf(max3f(m.x, m.y, m.z), m.w);
      const float r = mx == -CUDART_INF_F ? 0.0f : mx;
      auto part = [&](float mi, float si) { return si * ex2_approx((mi - r) * sl); };
      return Sums{mx, (part(m.x, s.x) + part(m.y, s.y)) + (part(m.z, s.z) + part(m.w, s.w)), 0.0f};
    } else {
      const int w = min(lane, kWarps - 1);
      return join_sums(kWarps, Sums{wmax[k & 1][w], wsum[k & 1][w], 0.0f}, sl);
    }
  };
  auto row_sums = [&](int k) {
    if (slices == 1) return block_sums(k);
    wait(&rec_bar[k & 1], k >> 1);
    const float* q = rec[k & 1][min(lane, slices - 1)];
    return join_sums(slices, Sums{q[0], q[1], 0.0f}, sl);
  };

  if (warp == kWarps) {
    // ---------------------------------------------------------------- teacher
    int2* raw = reinterpret_cast<int2*>(buffers + nbuf * buf_stride);   // all of the next row's
    int2* own_of[2] = {raw + a.K, raw + 2 * a.K};                      // the block's, by parity
    float* own_x = reinterpret_cast<float*>(raw + 3 * a.K);            // their logits
    float4 next_info = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto fetch = [&](int64_t t) {
#pragma unroll 4
      for (int s = lane; s < a.K; s += 32) copy_entry(&raw[s], &slots.entries[t * a.K + s]);
      next_info = slots.info[t];
    };
    // the block's own tokens of row t, in slot order; how many
    auto prepare = [&](int64_t t, int b) -> int {
      const RowShape<IT> shape(t * a.v, a.v);
      const int own0 = shape.head + min(rank * per, shape.units) * kN;
      const int own1 = shape.head + min(rank * per + per, shape.units) * kN;
      const int body1 = shape.head + shape.units * kN;
      if (lane == 0) row_info[b] = next_info;
      copy_wait();
      int n = 0;
#pragma unroll 4
      for (int s0 = 0; s0 < a.K; s0 += 32) {
        int2 e = make_int2(-1, 0);
        if (s0 + lane < a.K) e = raw[s0 + lane];
        const bool own = (e.x >= own0 && e.x < own1) ||
                         (rank == 0 && e.x >= 0 && (e.x < shape.head || e.x >= body1));
        const uint32_t mask = __ballot_sync(0xffffffffu, own);
        if (own) own_of[b][n + __popc(mask & ((1u << lane) - 1u))] = e;
        n += __popc(mask);
      }
      __syncwarp();
      return n;
    };

    grid_dependency_wait();   // the entries are there
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
      const int2* own = own_of[par];
      const IT* slice =
          reinterpret_cast<const IT*>(buffers + (nbuf == 2 ? par : 0) * buf_stride);
      if (rank == 0 && lane == 0 && slices > 1 && !late)
        mbar_arrive_expect_tx(&own_bar[par], static_cast<uint32_t>(slices) * 16u);
      wait_slice(k);
#pragma unroll 4
      for (int e = lane; e < n; e += 32) {
        const int id = own[e].x;
        own_x[e] = id >= own0 && id < own1
                       ? to_f32(slice[id - own0])
                       : to_f32(static_cast<const IT*>(a.logits)[t * a.v + id]);
      }
      named_barrier_sync(1, NT + 32);   // the slice has been read, the warps' sums are there
      const float block_m = block_sums(k).m;
      const float block_ref = block_m == -CUDART_INF_F ? 0.0f : block_m;
      float A = 0.0f, P_own = 0.0f;
#pragma unroll 4
      for (int e = lane; e < n; e += 32) {
        const float p = __int_as_float(own[e].y);
        A = fmaf(p, own_x[e] - block_ref, A);
        P_own += p;
      }
      A = warp_sum(A);
      P_own = warp_sum(P_own);
      if (slices > 1 && lane == 0 && !late)
        st_async_v4(mapa_shared(&own_rec[par][rank][0], 0), mapa_shared(&own_bar[par], 0), A, P_own,
                    block_ref, 0.0f);
      int n_next = 0;
      if (t + clusters < a.T) {
        n_next = prepare(t + clusters, par ^ 1);
        if (t + 2 * clusters < a.T) fetch(t + 2 * clusters);
      }
      const Sums all = row_sums(k);
      const float ref = all.m == -CUDART_INF_F ? 0.0f : all.m;
      const float4 info = row_info[par];
      const float P = info.x, w = info.w;
      const bool any_bad = info.z != 0.0f;
      const bool dead = w == 0.0f || (P == 0.0f && !any_bad);
      if (rank == 0) {
        if (slices > 1) {   // the slices' A moved to the common reference, in slice order
          wait(&own_bar[par], k >> 1);
          A = 0.0f;
          for (int i = 0; i < slices; ++i) {
            const float* q = own_rec[par][i];
            if (q[1] != 0.0f) A += fmaf(q[2] - ref, q[1], q[0]);
          }
        }
        if (lane == 0) {
          const float log_s = logf(all.s);
          const float loss = fmaf(P, log_s, fmaf(-a.scale, A, info.y));
          a.loss[t] = dead ? 0.0f : any_bad ? CUDART_NAN_F : w * loss;
          if (a.lse) a.lse[t] = fmaf(a.scale, ref, log_s);
          if (!dead && any_bad && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
        }
      }
      named_barrier_sync(2, NT + 32);   // P·q is written
      if (!dead) {
        const float c = any_bad ? CUDART_NAN_F : a.grad_scale * w * a.scale;
        const float inv = 1.0f / all.s;
        GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
#pragma unroll 4
        for (int e = lane; e < n; e += 32)
          put(out + own[e].x, c * (P * (ex2_approx((own_x[e] - ref) * sl) * inv) -
                                   __int_as_float(own[e].y)));
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
      if (t == stall_row && rank == 0) return;   // diagnostics: the copy never comes
      const char* src = static_cast<const char*>(a.logits) +
                        (t * a.v + shape.head) * static_cast<int64_t>(sizeof(IT)) +
                        static_cast<int64_t>(u0) * 16;
      uint8_t* dst = buffers + b * buf_stride;
      for (uint32_t off = 0; off < bytes; off += 16384u)
        bulk_load(dst + off, src + off, min(bytes - off, 16384u), &load_bar[b]);
    };
    if (tid == 32) {
      int n = 0;
      for (; n < nbuf && cluster + n * clusters < a.T; ++n) issue(n, cluster + n * clusters);
      asked = n;
    }
    constexpr uint32_t kInf = Unit<IT>::kMinusInf;
    const uint4 fill = make_uint4(kInf, kInf, kInf, kInf);
    // the row's edges: thread i of block 0 the i-th element of the head, thread
    // 32 + i of the tail; loaded a row ahead
    auto edge_of = [&](const RowShape<IT>& shape) {
      if (rank == 0 && tid < shape.head) return tid;
      if (rank == 0 && tid >= 32 && tid < 32 + shape.tail)
        return shape.head + shape.units * kN + tid - 32;
      return -1;
    };
    auto load_edge = [&](int64_t t) {
      const int j = t < a.T ? edge_of(RowShape<IT>(t * a.v, a.v)) : -1;
      return j >= 0 ? to_f32(static_cast<const IT*>(a.logits)[t * a.v + j]) : -CUDART_INF_F;
    };
    float next_edge = load_edge(cluster);
    int k = 0;
    for (int64_t t = cluster; t < a.T; t += clusters, ++k) {
      const int par = k & 1;
      const RowShape<IT> shape(t * a.v, a.v);
      const int u0 = min(rank * per, shape.units);
      const int n = min(u0 + per, shape.units) - u0;
      const uint4* slice =
          reinterpret_cast<const uint4*>(buffers + (nbuf == 2 ? par : 0) * buf_stride);
      // this row's records: one arrival here, 16 bytes from each slice
      if (tid == 0 && slices > 1 && !late)
        mbar_arrive_expect_tx(&rec_bar[par], static_cast<uint32_t>(slices) * 16u);
      const int my_edge = edge_of(shape);
      const float edge_x = next_edge;
      wait_slice(k);
      Held<IT, R> held;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int u = tid + i * NT;
        held.take(i, u < n ? slice[u] : fill);
      }
      const float m_w = warp_max(held.maximum(edge_x));
      const float ref_w = m_w == -CUDART_INF_F ? 0.0f : m_w;
      float s_w = held.sum(ref_w, sl);
      if (my_edge >= 0) s_w += ex2_approx((edge_x - ref_w) * sl);
      s_w = warp_sum(s_w);
      if (lane == 0) {
        wmax[par][warp] = m_w;
        wsum[par][warp] = s_w;
      }
      named_barrier_sync(1, NT + 32);
      if (tid == 32 && t + nbuf * clusters < a.T && !late) {
        fence_proxy_async_smem();
        issue(nbuf == 2 ? par : 0, t + nbuf * clusters);
        asked = k + nbuf + 1;
      }
      next_edge = load_edge(t + clusters);
      if (slices > 1 && warp == 0) {
        const Sums own = block_sums(k);
        if (lane < slices && !late)
          st_async_v4(mapa_shared(&rec[par][rank][0], static_cast<uint32_t>(lane)),
                      mapa_shared(&rec_bar[par], static_cast<uint32_t>(lane)), own.m, own.s, 0.0f,
                      0.0f);
      }
      const Sums all = row_sums(k);
      const float ref = all.m == -CUDART_INF_F ? 0.0f : all.m;
      const float4 info = row_info[par];
      const float P = info.x, w = info.w;
      const bool any_bad = info.z != 0.0f;
      const bool dead = w == 0.0f || (P == 0.0f && !any_bad);
      const float coef = any_bad ? CUDART_NAN_F : a.grad_scale * w * a.scale * (P * (1.0f / all.s));
      GT* out = static_cast<GT*>(a.dlogits) + t * a.v;
      GT* dst = out + shape.head + static_cast<int64_t>(u0) * kN;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int u = tid + i * NT;
        if (u < n) {
          float g[kN] = {};
          if (!dead) held.gradient(i, ref, sl, coef, g);
          put_unit<kN>(dst + static_cast<int64_t>(u) * kN, g);
        }
      }
      if (my_edge >= 0)
        put(out + my_edge, dead ? 0.0f : coef * ex2_approx((edge_x - ref) * sl));
      // the teacher warp's writes come after these; nothing here waits
      named_barrier_arrive(2, NT + 32);
    }
    if (tid == 32 && late)   // copies that may still be on their way into this block
      for (int r = max(asked - nbuf, 0); r < asked; ++r)
        mbar_wait_cluster_bounded(&load_bar[nbuf == 2 ? r & 1 : 0],
                                  static_cast<uint32_t>(nbuf == 2 ? r >> 1 : r) & 1u, wait_ns);
  }
  __syncthreads();
  if (slices > 1) cluster_sync_all();   // every peer's record into this block has landed
}

// One-shot debug injection (tp_debug_stall_next_distill) for the next launch.
std::mutex g_stall_mu;
int64_t g_stall_row = -1;
uint64_t g_stall_wait_ns = 0;
std::atomic<bool> g_stall_armed{false};

// One launch: rows in slices of `per` units.
template <typename IT, typename GT, int R, int NT>
tp_status launch(const DistillArgs& a, const Slots& slots, int slices, int per,
                 cudaStream_t stream) {
  // two buffers (rows ahead) while the blocks that the registers allow still
  // fit an SM, else one
  constexpr int kBlocks = blocks_per_sm(R, NT);
  constexpr int64_t kSmem = 224 * 1024 / kBlocks - 2048;   // a block's share, less its static part
  const int64_t stride = (static_cast<int64_t>(per) * 16 + 127) & ~int64_t{127};
  const int64_t lists = 28 * a.K;
  const int nbuf = 2 * stride + lists <= kSmem ? 2 : 1;
  const int smem = static_cast<int>(nbuf * stride + lists);
  auto kernel = distill_kernel<IT, GT, R, NT>;
  int dev = 0;
  cudaGetDevice(&dev);
  static bool configured[64] = {false};
  if (!configured[dev & 63]) {
    constexpr int64_t kMost = ((R * NT * 16 + 127) & ~127) + 28 * kDistillMaxK;
    static_assert(kMost <= 224 * 1024, "shared memory of one block");
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kMost > kSmem ? kMost : kSmem)) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess) {
      cudaGetLastError();
      return TP_ERR_CUDA;
    }
    configured[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NT + 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // programmatic dependent launch: the blocks set up and read their first
  // rows while the slots' kernel runs; only the teacher warps wait for it
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // clusters that can be resident at once, by launch shape
  struct Resident {
    int dev = -1, slices = 0, smem = 0, clusters = 0;
  };
  static thread_local Resident last;
  if (last.dev != dev || last.slices != slices || last.smem != smem) {
    int n = 0;
    cfg.gridDim = dim3(static_cast<unsigned>(slices * num_sms()));
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = num_sms() / slices;
    }
    last.dev = dev;
    last.slices = slices;
    last.smem = smem;
    last.clusters = n;
  }
  int64_t stall_row = -1;
  uint64_t wait_ns = wait_limit_ns();
  if (g_stall_armed.load(std::memory_order_relaxed)) {
    std::lock_guard<std::mutex> lk(g_stall_mu);
    if (g_stall_armed.exchange(false)) {
      stall_row = g_stall_row;
      wait_ns = g_stall_wait_ns;
    }
  }
  const int64_t clusters = a.T < last.clusters ? a.T : last.clusters;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * slices));
  if (cudaLaunchKernelEx(&cfg, kernel, a, slots, slices, per, nbuf, static_cast<uint32_t>(stride),
                         wait_ns, stall_row) != cudaSuccess) {
    cudaGetLastError();
    return TP_ERR_CUDA;
  }
  note_launches(1);
  return TP_OK;
}

template <typename IT, typename GT>
tp_status distill_launch_t(const DistillArgs& a, const Slots& slots, cudaStream_t stream) {
  constexpr int kN = Unit<IT>::kN;
  const int64_t units = (a.v + kN - 1) / kN;
  // Slices of a row: as few of 1, 2, 4, 6 and 8 as hold it.  A row of 50304 fp32
  // logits in gradient steps of 8192 rows takes 409 us on two blocks of 480
  // threads (411 on two of 512) and took 643 us on eight of 128: every exchange waits for the last of the
  // row's blocks.  Clusters have to fit the GPU's processing clusters: 22 of six
  // blocks are resident, 15 of eight, 26 of five and 45 of three, and 500 fp32
  // rows of 200001 took 137, 161 and 165 us on six, eight and five, 800 rows of
  // 100000 117 and 121 us on four and three.
  // With few rows, more slices while each keeps 4 KB.
  int slices = 1;
  for (;;) {
    const int next = slices < 4 ? 2 * slices : slices + 2;
    if (next > kMaxSlices) break;
    if (units <= 22 * 480 * slices &&
        !(a.T * next <= num_sms() && units * 16 >= 4096 * static_cast<int64_t>(next)))
      break;
    slices = next;
  }
  const int per = static_cast<int>((units + slices - 1) / slices);
  // Units a thread x streaming threads.  480 and the teacher's warp make 16 warps
  // on four schedulers, with 128 registers each (two blocks: 64); 512 make 17,
  // with 96 (56): 777 bf16 rows of 50257 take 40.8 us on 14 x 480, 42.2 on 13 x 512.
  // 9 x 480 spills at its 64 registers, fp32 to fp32 80 bytes a thread: 8192 rows of
  // 16000 take 188 us (138 to bf16, which spills 16).
  if (per <= 4 * 128) return launch<IT, GT, 4, 128>(a, slots, slices, per, stream);
  if (per <= 8 * 128) return launch<IT, GT, 8, 128>(a, slots, slices, per, stream);
  if (per <= 13 * 128) return launch<IT, GT, 13, 128>(a, slots, slices, per, stream);
  if (per <= 10 * 256) return launch<IT, GT, 10, 256>(a, slots, slices, per, stream);
  if (per <= 13 * 256) return launch<IT, GT, 13, 256>(a, slots, slices, per, stream);
  if (per <= 9 * 480) return launch<IT, GT, 9, 480>(a, slots, slices, per, stream);
  if (per <= 10 * 512) return launch<IT, GT, 10, 512>(a, slots, slices, per, stream);
  if (per <= 14 * 480) return launch<IT, GT, 14, 480>(a, slots, slices, per, stream);
  if (per <= 18 * 480) return launch<IT, GT, 18, 480>(a, slots, slices, per, stream);
  if (per <= 22 * 480) return launch<IT, GT, 22, 480>(a, slots, slices, per, stream);
  return TP_ERR_UNSUPPORTED;
}

}  // namespace

namespace {

// f(slots per lane) for K slots
template <typename F>
void with_slots(int K, F f) {
  if (K <= 32) f(std::integral_constant<int, 1>());
  else if (K <= 64) f(std::integral_constant<int, 2>());
  else if (K <= 128) f(std::integral_constant<int, 4>());
  else f(std::integral_constant<int, 8>());
}

}  // namespace

void arm_distill_stall(int64_t row, uint64_t wait_ns) {
  std::lock_guard<std::mutex> lk(g_stall_mu);
  g_stall_row = row;
  g_stall_wait_ns = wait_ns;
  g_stall_armed = true;
}

size_t distill_ws_bytes(int64_t T, int64_t K) {
  return static_cast<size_t>(T) * (sizeof(float4) + K * sizeof(int2));
}

tp_status distill_launch(const DistillArgs& a, tp_dtype dt, tp_dtype grad_dt, float* loss_sum,
                         void* ws, cudaStream_t stream) {
  static_assert(kDistillMaxK <= 8 * 32, "slots of a row in one warp");
  const unsigned prep = static_cast<unsigned>((a.T + kPrepWarps - 1) / kPrepWarps);
  if (a.dlogits == nullptr) {
    LogprobsArgs l = {};
    l.logits = a.logits;
    l.T = a.T;
    l.v = a.v;
    l.scale = a.scale;
    l.lse = a.lse;
    l.sums = static_cast<float2*>(ws);
    if (tp_status st = logprobs_fwd_launch(l, dt, stream)) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(prep);
    cfg.blockDim = dim3(kPrepWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t err = cudaSuccess;
    with_slots(a.K, [&](auto s) {
      err = dt == TP_DTYPE_BF16
                ? cudaLaunchKernelEx(&cfg, distill_loss_kernel<__nv_bfloat16, s()>, a,
                                     static_cast<const float2*>(l.sums))
                : cudaLaunchKernelEx(&cfg, distill_loss_kernel<float, s()>, a,
                                     static_cast<const float2*>(l.sums));
    });
    if (err != cudaSuccess) {
      cudaGetLastError();
      return TP_ERR_CUDA;
    }
    note_launches(1);
    return loss_sum ? loss_sum_launch(a.loss, a.T, loss_sum, stream, true) : TP_OK;
  }
  float4* info = static_cast<float4*>(ws);
  int2* entries = reinterpret_cast<int2*>(info + a.T);
  with_slots(a.K, [&](auto s) {
    distill_slots_kernel<s()><<<prep, kPrepWarps * 32, 0, stream>>>(a, entries, info);
  });
  note_launches(1);
  if (cudaGetLastError() != cudaSuccess) return TP_ERR_CUDA;
  const Slots slots{entries, info};
  const bool f32_grad = grad_dt == TP_DTYPE_F32;
  tp_status st;
  if (dt == TP_DTYPE_BF16)
    st = f32_grad ? distill_launch_t<__nv_bfloat16, float>(a, slots, stream)
                  : distill_launch_t<__nv_bfloat16, __nv_bfloat16>(a, slots, stream);
  else
    st = f32_grad ? distill_launch_t<float, float>(a, slots, stream)
                  : distill_launch_t<float, __nv_bfloat16>(a, slots, stream);
  if (st) return st;
  return loss_sum ? loss_sum_launch(a.loss, a.T, loss_sum, stream, true) : TP_OK;
}

}  // namespace tpl
