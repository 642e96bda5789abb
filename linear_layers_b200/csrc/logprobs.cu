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

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "rowwise.cuh"
#include "sm100_ptx.cuh"

namespace tpl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// ---------------------------------------------------------------------------
// top alternatives
// ---------------------------------------------------------------------------
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

// The r-th largest of the warp's keys (distinct but for 0), 0 if there are fewer.
__device__ __forceinline__ uint64_t warp_rth_key(uint64_t key, int r) {
  uint64_t best = 0;
  for (int i = 0; i < r; ++i) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
    const uint32_t lo = __reduce_max_sync(
        0xffffffffu, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
    best = (static_cast<uint64_t>(hi) << 32) | lo;
    if (key == best) key = 0;
  }
  return best;
}

// The row's top k, exactly, from one streaming pass.  While a block adds up
// its range it only notes the maximum of each thread's elements in each of
// (up to) kGroups stretches of the range.  Then
//   - the threshold: the smallest over the warps of the ceil(k/8)-th largest
//     of the lanes' maxima, a key that at least k elements reach;
//   - the groups whose maximum reaches it (about 1.5·k of them) are read again
//     from L2 and their elements at or above the threshold become candidates;
//   - if more than kLimit candidates have gathered (equal or ordered values),
//     the threshold is raised among them and the rest dropped.  The buffer has
//     room for kLimit and one more step of the whole block: it cannot overflow.
// Gathering while streaming instead, against a threshold from the first
// elements, cost 33 instructions per element of a v=50304 row at k = 64.
template <int kStep>
struct Candidates {
  static constexpr int kLimit = 512;
  static constexpr int kRoom = kLimit + kStep + 16;
  static constexpr int kGroups = 16;
  uint64_t key[kRoom];
  uint64_t warp_key[kWarps];
  uint64_t kth;
  float group_max[kGroups][kThreads];
  uint16_t hit[kGroups * kThreads];
  int n, kept, hits;

  // Smallest over the warps of the r-th largest key held by their lanes.
  __device__ __forceinline__ uint64_t threshold(uint64_t lane_key, int k) {
    const uint64_t w = warp_rth_key(lane_key, (k + kWarps - 1) / kWarps);
    if ((threadIdx.x & 31) == 0) warp_key[threadIdx.x >> 5] = w;
    __syncthreads();
    uint64_t t = warp_key[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) t = t < warp_key[i] ? t : warp_key[i];
    return t;
  }
  // Keeps the candidates that `keep(i, key)` accepts; all threads, after a
  // barrier.  Blocks of candidates move down in order: what a block writes
  // lies below what the later blocks read.
  template <typename F>
  __device__ __forceinline__ int compact(int count, F keep) {
    if (threadIdx.x == 0) kept = 0;
    for (int base = 0; base < count; base += kThreads) {
      const int i = base + static_cast<int>(threadIdx.x);
      const uint64_t q = i < count ? key[i] : 0;
      const bool ok = i < count && keep(i, q);
      __syncthreads();
      if (ok) key[atomicAdd(&kept, 1)] = q;
    }
    __syncthreads();
    const int left = kept;
    __syncthreads();
    return left;
  }
  // Fewer candidates, the top k among them; raises t.  All threads, after a
  // barrier; ends with one.
  __device__ __forceinline__ int shrink(int count, int k, uint64_t& t) {
    uint64_t best = 0;
    for (int i = threadIdx.x; i < count; i += kThreads) best = best > key[i] ? best : key[i];
    const uint64_t low = threshold(best, k);
    if (low > t) t = low;
    const uint64_t floor_key = t;
    return compact(count, [=](int, uint64_t q) { return q >= floor_key; });
  }
  // The same down to k exactly (count² / 256 comparisons a thread): for
  // orders of values that the threshold does not thin out.
  __device__ __forceinline__ int shrink_exact(int count, int k, uint64_t& t) {
    uint32_t flags = 0;
    static_assert((kRoom + kThreads - 1) / kThreads <= 32, "one flag per candidate of a thread");
    for (int i = threadIdx.x, b = 0; i < count; i += kThreads, ++b) {
      const uint64_t q = key[i];
      int rank = 0;
      for (int j = 0; j < count; ++j) rank += key[j] > q;
      if (rank < k) flags |= 1u << b;
      if (rank == k - 1) kth = q;
    }
    __syncthreads();
    const int left = compact(count, [=](int i, uint64_t) { return (flags >> (i / kThreads)) & 1u; });
    if (left == k && kth > t) t = kth;
    return left;
  }
};

// Log-probability statistics of one row by `slices` blocks (a cluster), each
// taking a contiguous range of the row's 16-byte units.  A block streams its
// range with the next step's loads in flight while it adds up the present
// one; sums and candidates of the blocks meet in block 0 through distributed
// shared memory.  Reading the row once is the bound: 256 threads hold 64 bytes
// each in flight.
template <typename IT, bool kTop>
__global__ void __launch_bounds__(kThreads, kTop ? 4 : 5)
    logprobs_kernel(const LogprobsArgs a, int slices) {
  constexpr int kN = Unit<IT>::kN;
  constexpr int kUnits = 2;                       // units per thread and step
  using Cand = Candidates<kTop ? kThreads * kN : 0>;
  extern __shared__ __align__(16) uint8_t dyn_smem[];
  Cand& cand = *reinterpret_cast<Cand*>(dyn_smem);   // only touched with kTop
  __shared__ Sums wsum[kWarps];
  __shared__ Sums bsum;
  __shared__ uint64_t best[kTop ? kLogprobsMaxK : 1];

  const int rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t t = blockIdx.x / static_cast<unsigned>(slices);
  const int64_t f0 = t * a.v;
  const RowShape<IT> shape(f0, a.v);
  const IT* row = static_cast<const IT*>(a.logits) + f0;
  const IT* body = row + shape.head;
  const int per = (shape.units + slices - 1) / slices;
  const int u0 = min(rank * per, shape.units), u1 = min(u0 + per, shape.units);
  const int tid = threadIdx.x;
  const float sl = a.scale * kLog2e;
  const float tau = 8.0f / sl;

  // the given token's logit, in flight behind the row
  int64_t y = -1;
  float xy = 0.0f;
  const bool want_y = rank == 0 && tid == 0 && a.targets != nullptr;
  if (want_y) {
    y = a.targets[t];
    if (y >= 0 && y < a.v) xy = to_f32(row[y]);
  }

  const uint4 fill = make_uint4(Unit<IT>::kMinusInf, Unit<IT>::kMinusInf, Unit<IT>::kMinusInf,
                                Unit<IT>::kMinusInf);
  auto load = [&](int base, uint4 (&w)[kUnits]) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = base + i * kThreads + tid;
      w[i] = u < u1 ? ld_unit(body + static_cast<int64_t>(u) * kN) : fill;
    }
  };
  // position in the row of unit u's first element
  auto first_of = [&](int u) { return static_cast<uint32_t>(shape.head + u * kN); };

  RowSums sums;
  uint4 next[kUnits];
  load(u0, next);
  const int steps = (u1 - u0 + kThreads * kUnits - 1) / (kThreads * kUnits);
  // steps per group, the group being filled, the lane's maximum and the last
  // position it can have (equal maxima: the first step's)
  [[maybe_unused]] const int group_steps = (steps + Cand::kGroups - 1) / Cand::kGroups;
  [[maybe_unused]] int group = 0, group_left = group_steps, lane_step = 0;
  [[maybe_unused]] float group_mx = -CUDART_INF_F, lane_mx = -CUDART_INF_F;
  [[maybe_unused]] bool lane_has = false;
  for (int st = 0; st < steps; ++st) {
    const int base = u0 + st * kThreads * kUnits;
    float x[kUnits * kN];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) Unit<IT>::unpack(next[i], x + i * kN);
    if (st + 1 < steps) load(base + kThreads * kUnits, next);
    const float mx = sums.add<kUnits * kN, true>(x, sl, tau);
    if constexpr (kTop) {
      if (st == 0) lane_has = u0 + tid < u1 && x[0] == x[0];
      if (mx > lane_mx) {
        lane_mx = mx;
        lane_step = st;
      }
      group_mx = fmaxf(group_mx, mx);
      if (--group_left == 0 || st + 1 == steps) {
        cand.group_max[group++][tid] = group_mx;
        group_mx = -CUDART_INF_F;
        group_left = group_steps;
      }
    }
  }
  // the edges of the row: at most kN − 1 elements at each end
  int edge_j = -1;
  float edge_x = 0.0f;
  if (rank == 0 && tid < shape.head) edge_j = tid;
  if (rank == slices - 1 && tid >= 32 && tid < 32 + shape.tail)
    edge_j = static_cast<int>(first_of(shape.units)) + tid - 32;
  if (edge_j >= 0) {
    edge_x = to_f32(row[edge_j]);
    sums.add1<true>(edge_x, sl, tau);
  }

  if constexpr (kTop) {
    bool full = false;   // a candidate landed at or past kLimit
    auto admit = [&](uint64_t q) {
      const int at = atomicAdd(&cand.n, 1);
      cand.key[at] = q;
      full |= at >= Cand::kLimit;
    };
    if (tid == 0) cand.n = cand.hits = 0;
    // A lane's key may place its maximum too late, never too early.  A lane
    // of nothing but −inf (or NaN) has its first element, if that is −inf.
    uint64_t lane_key = 0;
    if (lane_mx > -CUDART_INF_F)
      lane_key = rank_key(lane_mx, first_of(u0 + (lane_step * kUnits + kUnits - 1) * kThreads + tid) + kN - 1);
    else if (lane_has)
      lane_key = rank_key(-CUDART_INF_F, first_of(u0 + tid));
    uint64_t floor_key = cand.threshold(lane_key, a.top_k);   // a barrier within
    for (int g = 0; g < group; ++g) {
      const uint32_t at = first_of(u0 + g * group_steps * kUnits * kThreads + tid);
      if (rank_key(cand.group_max[g][tid], at) >= floor_key)
        cand.hit[atomicAdd(&cand.hits, 1)] = static_cast<uint16_t>(g * kThreads + tid);
    }
    if (edge_j >= 0 && edge_x == edge_x) {
      const uint64_t q = rank_key(edge_x, static_cast<uint32_t>(edge_j));
      if (q >= floor_key) admit(q);
    }
    __syncthreads();
    // one unit of a hit group per thread and round
    const int group_units = group_steps * kUnits;
    const int items = cand.hits * group_units;
    for (int base = 0; base < items; base += kThreads) {
      const int item = base + tid;
      if (item < items) {
        const int h = cand.hit[item / group_units];
        const int u = u0 + ((h / kThreads) * group_units + item % group_units) * kThreads +
                      h % kThreads;
        if (u < u1) {
          float x[kN];
          Unit<IT>::unpack(*reinterpret_cast<const uint4*>(body + static_cast<int64_t>(u) * kN), x);
          const float floor_x = floor_key ? key_value(floor_key) : -CUDART_INF_F;
#pragma unroll
          for (int i = 0; i < kN; ++i)
            if (x[i] >= floor_x) {   // not NaN
              const uint64_t q = rank_key(x[i], first_of(u) + i);
              if (q >= floor_key) admit(q);
            }
        }
      }
      if (__syncthreads_or(full)) {
        int left = cand.shrink(cand.n, a.top_k, floor_key);
        if (left > Cand::kLimit / 2) left = cand.shrink_exact(left, a.top_k, floor_key);
        full = false;
        if (tid == 0) cand.n = left;
        __syncthreads();
      }
    }
  }

  const Sums w = warp_sums(sums, sl);
  if ((tid & 31) == 0) wsum[tid >> 5] = w;
  __syncthreads();
  Sums all = join_sums(kWarps, wsum[min(tid & 31, kWarps - 1)], sl);

  // this block's best: a count of the candidates, rank by rank
  [[maybe_unused]] auto ranked = [&](int n, auto&& out) {
    if constexpr (kTop) {
      uint64_t floor_key = 0;
      if (n > 2 * a.top_k + 64) n = cand.shrink(n, a.top_k, floor_key);
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t q = cand.key[i];
        int rank_of = 0;
        for (int j = 0; j < n; ++j) rank_of += cand.key[j] > q;
        if (rank_of < a.top_k) out(rank_of, q);
      }
      for (int i = n + tid; i < a.top_k; i += kThreads) out(i, 0);   // slots nothing fills
    }
  };
  if (slices > 1) {
    if constexpr (kTop) ranked(cand.n, [&](int i, uint64_t q) { best[i] = q; });
    if (tid == 0) bsum = all;
    cluster_sync_all();
    if (rank == 0) {
      const uint32_t at =
          mapa_shared(&bsum, static_cast<uint32_t>(min(tid & 31, slices - 1)));
      Sums q;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q.m) : "r"(at));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q.s) : "r"(at + 4));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q.u) : "r"(at + 8));
      all = join_sums(slices, q, sl);
      if constexpr (kTop) {
        if (tid == 0) cand.n = 0;
        __syncthreads();
        for (int i = tid; i < slices * a.top_k; i += kThreads) {
          uint64_t q;
          asm volatile("ld.shared::cluster.u64 %0, [%1];"
                       : "=l"(q)
                       : "r"(mapa_shared(&best[i % a.top_k], static_cast<uint32_t>(i / a.top_k))));
          if (q) cand.key[atomicAdd(&cand.n, 1)] = q;   // at most 8·128 of them
        }
        __syncthreads();
      }
    }
    cluster_sync_all();   // the peers' shared memory has been read
    if (rank != 0) return;
  }

  const float ref = all.m == -CUDART_INF_F ? 0.0f : all.m;
  const float log_s = logf(all.s);
  if (want_y) {
    const bool ok = y >= 0 && y < a.v;
    if (!ok && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
    if (a.logprob) a.logprob[t] = ok ? fmaf(a.scale, xy - ref, -log_s) : CUDART_NAN_F;
  }
  if (tid == 0) {
    if (a.entropy) a.entropy[t] = log_s - a.scale * (all.u / all.s);
    if (a.lse) a.lse[t] = fmaf(a.scale, ref, log_s);
    if (a.sums) a.sums[t] = make_float2(ref, log_s);
  }
  if constexpr (kTop)
    ranked(cand.n, [&](int i, uint64_t q) {
      const int64_t o = t * a.top_k + i;
      a.top_idx[o] = q ? key_index(q) : -1;
      a.top_logprob[o] = q ? fmaf(a.scale, key_value(q) - ref, -log_s) : CUDART_NAN_F;
    });
}

// Gradient of (log-probability, entropy): one pass over the logits, each
// block a contiguous range of one row, every thread's loads of its (up to)
// four units in flight at once.
constexpr int kBwdUnits = 4;

template <typename IT, typename GT>
__global__ void __launch_bounds__(kThreads) logprobs_bwd_kernel(const LogprobsBwdArgs a, int blocks) {
  constexpr int kN = Unit<IT>::kN;
  const int64_t t = blockIdx.x / static_cast<unsigned>(blocks);
  const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(blocks));
  const int64_t f0 = t * a.v;
  const RowShape<IT> shape(f0, a.v);
  const IT* row = static_cast<const IT*>(a.logits) + f0;
  GT* out = static_cast<GT*>(a.dlogits) + f0;
  const int per = (shape.units + blocks - 1) / blocks;
  const int u0 = min(part * per, shape.units), u1 = min(u0 + per, shape.units);
  const int tid = threadIdx.x;
  const float g = a.dlogprob ? a.dlogprob[t] : 0.0f;
  const float e = a.dentropy ? a.dentropy[t] : 0.0f;
  const bool zero = g == 0.0f && e == 0.0f;   // a padded row: nothing of it is read
  uint4 w[kBwdUnits];
#pragma unroll
  for (int i = 0; i < kBwdUnits; ++i) {
    const int u = u0 + i * kThreads + tid;
    w[i] = !zero && u < u1 ? ld_unit(row + shape.head + static_cast<int64_t>(u) * kN)
                           : make_uint4(0, 0, 0, 0);
  }
  int64_t y = -1;
  float bad = 0.0f, lse = 0.0f, h = 0.0f;
  if (!zero) {
    if (g != 0.0f) {
      y = a.targets[t];
      if (y < 0 || y >= a.v) {
        bad = CUDART_NAN_F;
        if (part == 0 && tid == 0 && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
      }
    }
    lse = a.lse[t];
    if (e != 0.0f) h = a.entropy[t];
  }
  const float geh = fmaf(e, h, g);
  // scale·(g·[j = y] − p·(g + e·(lp + h))), lp = scale·x − lse, p = exp(lp)
  auto grad = [&](float x, bool at_y) {
    const float lp = fmaf(x, a.scale, -lse);
    const float p = ex2_approx(lp * kLog2e);
    const float d = (at_y ? g : 0.0f) - p * fmaf(e, max_nan(lp, kLowest), geh);
    return zero ? 0.0f : fmaf(a.scale, d, bad);
  };
#pragma unroll
  for (int i = 0; i < kBwdUnits; ++i) {
    const int u = u0 + i * kThreads + tid;
    if (u >= u1) break;
    const int64_t j0 = shape.head + static_cast<int64_t>(u) * kN;
    const int at = static_cast<int>(min(max(y - j0, static_cast<int64_t>(-1)), static_cast<int64_t>(kN)));
    float x[kN];
    Unit<IT>::unpack(w[i], x);
#pragma unroll
    for (int q = 0; q < kN; ++q) x[q] = grad(x[q], q == at);
    put_unit<kN>(out + j0, x);
  }
  auto edge = [&](int64_t j) { put(out + j, grad(zero ? 0.0f : to_f32(row[j]), j == y)); };
  if (part == 0 && tid < shape.head) edge(tid);
  if (part == blocks - 1 && tid >= 32 && tid < 32 + shape.tail)
    edge(shape.head + static_cast<int64_t>(shape.units) * kN + tid - 32);
}

// Combine of the per-slice statistics of the output-layer GEMM (slice k of
// row t at [k·T + t]): M = max m_k, w_k = exp(scale·(m_k − M)),
// S = Σ w_k·s_k, U = Σ w_k·(u_k + (m_k − M)·s_k).  A block takes eight tokens
// (a 32-byte sector of each slice's row of numbers) and 32 slices at a time;
// the partial results meet in a fixed order.  One token per lane and eight
// slices at a time took 25 us of a T = 500, v = 50304 call, this takes 4.
constexpr int kCombTokens = 8;
constexpr int kCombSlices = kThreads / kCombTokens;

__global__ void __launch_bounds__(kThreads)
    linear_logprobs_combine_kernel(const float* __restrict__ stat_m,
                                   const float* __restrict__ stat_s,
                                   const float* __restrict__ stat_u,
                                   const float* __restrict__ tgt_logit,
                                   const int64_t* __restrict__ targets, int64_t T, int64_t v,
                                   int nslices, float scale, float* __restrict__ logprob,
                                   float* __restrict__ entropy, float* __restrict__ lse,
                                   int32_t* dev_status) {
  __shared__ float part_m[kWarps][kCombTokens];
  __shared__ float part_s[kWarps][kCombTokens];
  __shared__ float part_u[kWarps][kCombTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = lane & (kCombTokens - 1);
  const int first = threadIdx.x / kCombTokens;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kCombTokens + tok;
  const bool ok = t < T;
  float m = -CUDART_INF_F;
  if (ok) {
#pragma unroll 8
    for (int k = first; k < nslices; k += kCombSlices) m = fmaxf(m, stat_m[k * T + t]);
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
  if (lane < kCombTokens) part_m[warp][tok] = m;
  __syncthreads();
  float M = part_m[0][tok];
#pragma unroll
  for (int q = 1; q < kWarps; ++q) M = fmaxf(M, part_m[q][tok]);
  if (M == -CUDART_INF_F) M = 0.0f;   // nothing but −inf (or NaN) in the row
  float S = 0.0f, U = 0.0f;
  if (ok) {
#pragma unroll 4
    for (int k = first; k < nslices; k += kCombSlices) {
      const float d = stat_m[k * T + t] - M;
      const float f = ex2_approx(d * (scale * kLog2e));
      const float s = stat_s[k * T + t];
      S = fmaf(s, f, S);
      U = fmaf(f, fmaf(fmaxf(d, kLowest), s, stat_u[k * T + t]), U);
    }
  }
#pragma unroll
  for (int off = 8; off <= 16; off <<= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, off);
    U += __shfl_xor_sync(0xffffffffu, U, off);
  }
  if (lane < kCombTokens) {
    part_s[warp][tok] = S;
    part_u[warp][tok] = U;
  }
  __syncthreads();
  if (threadIdx.x < kCombTokens && ok) {
    S = 0.0f;
    U = 0.0f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      S += part_s[q][tok];
      U += part_u[q][tok];
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

namespace {

template <typename IT, bool kTop>
tp_status logprobs_fwd_launch_t(const LogprobsArgs& a, cudaStream_t stream) {
  // Blocks per row: one once the rows alone fill the GPU's resident blocks,
  // else up to eight (the portable cluster size) while each keeps a step or
  // more of the row.
  const int64_t units = a.v / Unit<IT>::kN;
  int slices = 1;
  while (slices < 8 && a.T * slices * 2 <= 4 * num_sms() && units / (slices * 2) >= 2 * kThreads)
    slices *= 2;
  constexpr size_t smem = kTop ? sizeof(Candidates<kThreads * Unit<IT>::kN>) : 0;
  static_assert(smem <= 48 * 1024, "within the default limit of dynamic shared memory");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T * slices));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = slices > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, logprobs_kernel<IT, kTop>, a, slices) != cudaSuccess) {
    cudaGetLastError();
    return TP_ERR_CUDA;
  }
  note_launches(1);
  return TP_OK;
}

template <typename IT, typename GT>
tp_status logprobs_bwd_launch_t(const LogprobsBwdArgs& a, cudaStream_t stream) {
  const int64_t units = a.v / Unit<IT>::kN;
  const int64_t blocks = units > 0 ? (units + kThreads * kBwdUnits - 1) / (kThreads * kBwdUnits) : 1;
  if (a.T * blocks > 0x7fffffff) return TP_ERR_UNSUPPORTED;   // more logits than any GPU holds
  logprobs_bwd_kernel<IT, GT><<<static_cast<unsigned>(a.T * blocks), kThreads, 0, stream>>>(
      a, static_cast<int>(blocks));
  note_launches(1);
  return last_error();
}

}  // namespace

tp_status logprobs_fwd_launch(const LogprobsArgs& a, tp_dtype dt, cudaStream_t stream) {
  if (dt == TP_DTYPE_BF16)
    return a.top_k ? logprobs_fwd_launch_t<__nv_bfloat16, true>(a, stream)
                   : logprobs_fwd_launch_t<__nv_bfloat16, false>(a, stream);
  return a.top_k ? logprobs_fwd_launch_t<float, true>(a, stream)
                 : logprobs_fwd_launch_t<float, false>(a, stream);
}

tp_status logprobs_bwd_launch(const LogprobsBwdArgs& a, tp_dtype dt, tp_dtype grad_dt,
                              cudaStream_t stream) {
  if (dt == TP_DTYPE_BF16)
    return grad_dt == TP_DTYPE_BF16 ? logprobs_bwd_launch_t<__nv_bfloat16, __nv_bfloat16>(a, stream)
                                    : logprobs_bwd_launch_t<__nv_bfloat16, float>(a, stream);
  return grad_dt == TP_DTYPE_BF16 ? logprobs_bwd_launch_t<float, __nv_bfloat16>(a, stream)
                                  : logprobs_bwd_launch_t<float, float>(a, stream);
}

tp_status linear_logprobs_combine_launch(const float* stat_m, const float* stat_s,
                                         const float* stat_u, const float* tgt_logit,
                                         const int64_t* targets, int64_t T, int64_t v, float scale,
                                         float* logprob, float* entropy, float* lse,
                                         int32_t* dev_status, cudaStream_t stream) {
  const int nslices = static_cast<int>((v + kXentSlice - 1) / kXentSlice);
  linear_logprobs_combine_kernel<<<static_cast<unsigned>((T + kCombTokens - 1) / kCombTokens),
                                   kThreads, 0, stream>>>(stat_m, stat_s, stat_u, tgt_logit, targets, T, v,
                                             nslices, scale, logprob, entropy, lse, dev_status);
  note_launches(1);
  return last_error();
}

}  // namespace tpl
