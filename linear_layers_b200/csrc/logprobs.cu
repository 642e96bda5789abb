// logprobs.cu — log-probabilities of given tokens, entropy and top
// alternatives of vocabulary-parallel logits, and their gradient.
//
//   z = scale·x,  M = max x,  S = Σ exp(scale·(x − M)),
//   U = Σ exp(scale·(x − M))·(x − M)
//   lse = scale·M + log S,  logprob = scale·(x_y − M) − log S,
//   entropy = log S − scale·U/S
//
// The sums run on differences to a reference near the maximum (within 1.4 of it
// in z), so that a large common offset of a row costs no bits, and an entropy's
// error is that of sums of size one, whatever the logits: about 2^-24 for each
// addition of a thread at worst, 6e-7 of an entropy of 0.75 as measured.
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

constexpr int kThreads = 128;       // of a forward block
constexpr int kWarps = kThreads / 32;
constexpr int kBwdThreads = 256;    // of a gradient block, and of the slices' combine
constexpr int kBwdWarps = kBwdThreads / 32;

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
constexpr uint32_t kBehind = 0x40000001u;   // behind every index
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int32_t key_index(uint64_t key) {
  return static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key));
}

// The r-th largest of the warp's keys, two per lane (key >= second; distinct but
// for 0), 0 if there are fewer.
__device__ __forceinline__ uint64_t warp_rth_key(uint64_t key, uint64_t second, int r) {
  uint64_t best = 0;
  for (int i = 0; i < r; ++i) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
    const uint32_t lo = __reduce_max_sync(
        0xffffffffu, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
    best = (static_cast<uint64_t>(hi) << 32) | lo;
    if (key == best) {
      key = second;
      second = 0;
    }
  }
  return best;
}

// The row's top k, exactly, from one streaming pass.  While a block adds up
// its range it notes the maximum of every group, the elements of one thread in
// one or few steps.  Then
//   - the threshold: the smallest over the warps of the ceil(k/4)-th largest
//     of their lanes' two largest maxima, a key that at least k elements reach;
//   - the groups whose maximum reaches it (about 1.5·k of them) are read again
//     and their elements at or above the threshold become candidates;
//   - the candidates are placed by counting.
// If more elements reach the threshold than the buffer holds (equal values),
// the range is read once more in barrier-separated steps, and whenever kLimit
// candidates have gathered the threshold is raised among them and the rest
// dropped.
// 8192 bf16 rows of 50304 take 139 us without alternatives, 164 at k = 1, 218 at
// k = 64, 296 at k = 128: what is behind a row's last load, with no load of that
// block in flight.  Gathering
// while streaming, against a threshold from the first elements, took twice the
// instructions.
struct Candidates {
  static constexpr int kLimit = 512;
  static constexpr int kRoom = kLimit + kThreads * 8 + 16;   // kLimit and a step of units
  static constexpr int kGroups = 32;
  static constexpr int kHits = 1024;
  uint64_t key[kRoom];
  uint64_t warp_key[kWarps];
  uint64_t kth;
  int n, kept;
  int hits;
  uint16_t hit[kHits];
  alignas(16) float4 group_max[];   // [groups / 4][kThreads], four groups each

  // Smallest over the warps of the ceil(k / kWarps)-th largest of the keys held
  // by their lanes, two each (a >= b).
  __device__ __forceinline__ uint64_t threshold(uint64_t key_a, uint64_t key_b, int k) {
    const uint64_t w = warp_rth_key(key_a, key_b, (k + kWarps - 1) / kWarps);
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
    uint64_t best = 0, second = 0;
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const uint64_t q = key[i];
      second = q > best ? best : q > second ? q : second;
      best = q > best ? q : best;
    }
    const uint64_t low = threshold(best, second, k);
    if (low > t) t = low;
    const uint64_t floor_key = t;
    return compact(count, [=](int, uint64_t q) { return q >= floor_key; });
  }
  // The same down to k exactly (count² / kThreads comparisons a thread): for
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

constexpr int kUnits = 4;           // 16-byte units per thread and step

// Log-probability statistics of one row by `slices` blocks (a cluster), each
// taking a contiguous range of the row's 16-byte units.  A block streams its
// range with the next step's loads in flight while it adds up the present
// one; sums and candidates of the blocks meet in block 0 through distributed
// shared memory.  Reading the row once is the bound for fp32 logits: 8192 rows
// of 50304 take 233 us, 7.1 TB/s, with four units a thread and step on eight
// blocks per SM (two units on ten: 241 us, and 82 against 63 us for 2048 rows,
// whose last wave has few blocks to keep loads in flight).  bf16 logits take as
// many instructions for half the bytes: 139 us, 5.9 TB/s.  The bf16 kernel with
// alternatives spills 4 bytes a thread at 72 registers.
template <typename IT, bool kTop>
__global__ void __launch_bounds__(kThreads, Unit<IT>::kN == 4 ? 8 : 7)
    logprobs_kernel(const LogprobsArgs a, int slices, int group_log) {
  constexpr int kN = Unit<IT>::kN;
  using Cand = Candidates;
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
  const Part part(shape.units, rank, slices);
  const int u0 = part.first, u1 = part.last;
  const int tid = threadIdx.x;
  const float sl = a.scale * kLog2e;
  const float tau = 2.0f / sl;   // how far a logit may exceed its reference
  if (a.sums) grid_dependents_launch();   // the distillation loss follows

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
    const IT* p = body + static_cast<int64_t>(base + tid) * kN;
    if (base + kThreads * kUnits <= u1) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) w[i] = ld_unit(p + i * kThreads * kN);
    } else {
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        w[i] = base + i * kThreads + tid < u1 ? ld_unit(p + i * kThreads * kN) : fill;
    }
  };
  // position in the row of unit u's first element
  auto first_of = [&](int u) { return static_cast<uint32_t>(shape.head + u * kN); };

  RowSums sums;
  uint4 next[kUnits];
  load(u0, next);
  const int steps = steps_of(u1 - u0, kThreads * kUnits);
  // Without alternatives a row of few steps does not repay the warp's common
  // reference: 30000 bf16 rows of 2048 (one step) took 81.6 us with it, 76.4
  // without.  With them it always does: top 8 of 16384 bf16 rows of 8192 (two steps)
  // 119.5 and 121.8 us, top 64 of 8192 bf16 rows of 50304 226 and 244.
  if (kTop || steps > 2) {
    float x[kN];
    Unit<IT>::unpack(next[0], x);
    sums.start(x, tau);
  }
  // groups of 2^group_log steps: no more than the launch has room for, whose
  // group_log is the widest block's
  const int group_steps = kTop ? 1 << group_log : max(steps, 1);
  const int groups = kTop ? groups_of(steps, group_log) : min(steps, 1);
  [[maybe_unused]] bool lane_has = false;   // the lane's first element is there and a number
  if constexpr (kTop) {
    float x[kN];
    Unit<IT>::unpack(next[0], x);
    lane_has = u0 + tid < u1 && x[0] == x[0];
  }
  int st = 0;
  for (int g = 0; g < groups; ++g) {
    [[maybe_unused]] float group_mx = -CUDART_INF_F;
    const int end = min(st + group_steps, steps);
    for (; st < end; ++st) {
      float x[kUnits * kN];
#pragma unroll
      for (int i = 0; i < kUnits; ++i) Unit<IT>::unpack(next[i], x + i * kN);
      if (st + 1 < steps) load(u0 + (st + 1) * kThreads * kUnits, next);
      const float mx = sums.add<kUnits * kN, true>(x, sl, tau);
      if constexpr (kTop) group_mx = fmaxf(group_mx, mx);
    }
    if constexpr (kTop)
      reinterpret_cast<float*>(&cand.group_max[(g >> 2) * kThreads + tid])[g & 3] = group_mx;
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
    if (tid == 0) cand.n = cand.hits = 0;
    // what the last four groups have of places without a group
    for (int g = groups; g & 3; ++g)
      reinterpret_cast<float*>(&cand.group_max[(g >> 2) * kThreads + tid])[g & 3] = -CUDART_INF_F;
    const int quads = (groups + 3) >> 2;
    float mx_a = -CUDART_INF_F, mx_b = -CUDART_INF_F;   // the lane's two largest maxima
    auto with_max = [&](float gm) {
      mx_b = fmaxf(mx_b, fminf(mx_a, gm));
      mx_a = fmaxf(mx_a, gm);
    };
    for (int q = 0; q < quads; ++q) {
      const float4 m4 = cand.group_max[q * kThreads + tid];
      with_max(m4.x);
      with_max(m4.y);
      with_max(m4.z);
      with_max(m4.w);
    }
    // The keys place the maxima behind every element of the row (a threshold
    // may be low, never high), apart from each other.  A lane of nothing but
    // −inf (or NaN) has its first element, if that is −inf.
    uint64_t key_a = 0, key_b = 0;
    if (mx_a > -CUDART_INF_F)
      key_a = rank_key(mx_a, kBehind + 2 * tid);
    else if (lane_has)
      key_a = rank_key(-CUDART_INF_F, first_of(u0 + tid));
    if (mx_b > -CUDART_INF_F) key_b = rank_key(mx_b, kBehind + 2 * tid + 1);
    uint64_t floor_key = cand.threshold(key_a, key_b, a.top_k);   // a barrier within
    // a place in a list of the block for each of the warp's lanes' n entries
    auto places = [&](int n, int* total) {
      int upto = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, off);
        if ((tid & 31) >= off) upto += o;
      }
      int base = 0;
      if ((tid & 31) == 31 && upto) base = atomicAdd(total, upto);
      return __shfl_sync(0xffffffffu, base, 31) + upto - n;
    };
    auto fetch = [&](int u) {
      return u < u1 ? *reinterpret_cast<const uint4*>(body + static_cast<int64_t>(u) * kN) : fill;
    };
    auto admit_edge = [&]() {
      if (edge_j >= 0 && edge_x == edge_x) {
        const uint64_t q = rank_key(edge_x, static_cast<uint32_t>(edge_j));
        if (q >= floor_key) cand.key[atomicAdd(&cand.n, 1)] = q;   // the first few places
      }
    };
    admit_edge();
    const float floor_x = floor_key ? key_value(floor_key) : -CUDART_INF_F;
    const uint32_t floor_at = static_cast<uint32_t>(key_index(floor_key));
    if (floor_key) {
      uint32_t hits = 0;   // bit g: group g of this thread reaches it
      for (int q = 0; q < quads; ++q) {
        const float4 m4 = cand.group_max[q * kThreads + tid];
        hits |= ((m4.x >= floor_x ? 1u : 0u) | (m4.y >= floor_x ? 2u : 0u) |
                 (m4.z >= floor_x ? 4u : 0u) | (m4.w >= floor_x ? 8u : 0u)) << (4 * q);
      }
      if (floor_x == -CUDART_INF_F) {
        // few elements above −inf, and the first ones of −inf: of the groups of
        // nothing else only those that begin no later than the threshold's place
        for (uint32_t h = hits; h; h &= h - 1) {
          const int g = __ffs(h) - 1;
          if (reinterpret_cast<const float*>(&cand.group_max[(g >> 2) * kThreads + tid])[g & 3] == floor_x &&
              first_of(u0 + g * group_steps * kUnits * kThreads + tid) > floor_at)
            hits &= ~(1u << g);
        }
      }
      for (int at = places(__popc(hits), &cand.hits); hits; hits &= hits - 1, ++at)
        if (at < Cand::kHits)
          cand.hit[at] = static_cast<uint16_t>((__ffs(hits) - 1) * kThreads + tid);
      __syncthreads();
      // one unit of a hit group per thread
      const int group_units = group_steps * kUnits;
      const int items = min(cand.hits, Cand::kHits) * group_units;
      for (int first = tid & ~31; first < items; first += kThreads) {   // warp by warp
        const int item = first + (tid & 31);
        int u = u1;
        if (item < items) {
          const int h = cand.hit[item / kUnits >> group_log];
          u = u0 + ((h / kThreads) * group_units + (item & (group_units - 1))) * kThreads + h % kThreads;
        }
        float x[kN];
        Unit<IT>::unpack(fetch(u), x);
        // above the threshold's value, or equal and no later
        const uint32_t first_at = u < u1 ? first_of(u) : 0xffffff00u;
        uint32_t take = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (x[i] > floor_x || (x[i] == floor_x && first_at + i <= floor_at)) take |= 1u << i;
        int at = places(__popc(take), &cand.n);
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if ((take >> i) & 1u) {
            if (at < Cand::kRoom) cand.key[at] = rank_key(x[i], first_at + i);
            ++at;
          }
      }
    }
    __syncthreads();
    if (!floor_key || cand.n > Cand::kRoom || cand.hits > Cand::kHits) {
      // fewer lanes with elements than a threshold needs, or more elements
      // that reach it than there is room for: the whole range again, step by
      // step, by value and place
      __syncthreads();
      if (tid == 0) cand.n = 0;
      __syncthreads();
      admit_edge();
      __syncthreads();
      for (int base = u0; base < u1; base += kThreads) {
        const int u = base + tid;
        float x[kN];
        Unit<IT>::unpack(fetch(u), x);
        uint32_t take = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (u < u1 && x[i] == x[i] && rank_key(x[i], first_of(u) + i) >= floor_key) take |= 1u << i;
        int at = places(__popc(take), &cand.n);
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if ((take >> i) & 1u) cand.key[at++] = rank_key(x[i], first_of(u) + i);
        if (__syncthreads_or(at > Cand::kLimit)) {
          int left = cand.shrink(cand.n, a.top_k, floor_key);
          if (left > Cand::kLimit / 2) left = cand.shrink_exact(left, a.top_k, floor_key);
          if (tid == 0) cand.n = left;
          __syncthreads();
        }
      }
    }
  }

  const Sums w = warp_sums(sums, sl);
  if ((tid & 31) == 0) wsum[tid >> 5] = w;
  __syncthreads();
  Sums all = join_sums(kWarps, wsum[min(tid & 31, kWarps - 1)], sl);

  // the top k of the n candidates, each placed by how many lie above it
  [[maybe_unused]] auto ranked = [&](int n, auto&& out) {
    if constexpr (kTop) {
      uint64_t floor_key = 0;
      if (n > 3 * a.top_k + 64) n = cand.shrink(n, a.top_k, floor_key);
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t q = cand.key[i];
        int rank_of = 0;
        const ulonglong2* two = reinterpret_cast<const ulonglong2*>(cand.key);
#pragma unroll 4
        for (int j = 0; j < n / 2; ++j) {
          const ulonglong2 o = two[j];
          rank_of += (o.x > q) + (o.y > q);
        }
        if (n & 1) rank_of += cand.key[n - 1] > q;
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

// Gradient of (log-probability, entropy), with lp = scale·x − lse and p = exp(lp):
//   scale·(g·[j = y] − p·(g + e·(lp + h))) = p·(e'·lp + c) + [j = y]·scale·g,
//   e' = −scale·e,  c = −scale·(g + e·h)
// One pass over the logits, bound by their bytes and the gradient's: each block
// a contiguous range of one row, every thread's loads of its (up to) four
// units in flight at once.  8192 rows of 50304, fp32 to bf16, one row in eight
// padded (written as zeros, not read): 335 us, 6.8 TB/s; on single elements
// instead of packed pairs the same took 396 us.
constexpr int kBwdUnits = 4;

template <typename IT, typename GT>
__global__ void __launch_bounds__(kBwdThreads) logprobs_bwd_kernel(const LogprobsBwdArgs a, int blocks) {
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
  // this thread's edge element, if any
  int edge = -1;
  if (part == 0 && tid < shape.head) edge = tid;
  if (part == blocks - 1 && tid >= 32 && tid < 32 + shape.tail)
    edge = shape.head + shape.units * kN + tid - 32;
  const float g = a.dlogprob ? a.dlogprob[t] : 0.0f;
  const float e = a.dentropy ? a.dentropy[t] : 0.0f;
  if (g == 0.0f && e == 0.0f) {   // a padded row: nothing of it is read
    const float z[kN] = {};
    for (int u = u0 + tid; u < u1; u += kBwdThreads)
      put_unit<kN>(out + shape.head + static_cast<int64_t>(u) * kN, z);
    if (edge >= 0) put(out + edge, 0.0f);
    return;
  }
  uint4 w[kBwdUnits];
#pragma unroll
  for (int i = 0; i < kBwdUnits; ++i) {
    const int u = u0 + i * kBwdThreads + tid;
    w[i] = u < u1 ? ld_unit(row + shape.head + static_cast<int64_t>(u) * kN) : make_uint4(0, 0, 0, 0);
  }
  const float edge_x = edge >= 0 ? to_f32(row[edge]) : 0.0f;
  int64_t y = -1;
  float c = -a.scale * g;
  const float e1 = -a.scale * e;
  if (g != 0.0f) {
    y = a.targets[t];
    if (y < 0 || y >= a.v) {
      c = CUDART_NAN_F;   // the whole row
      if (part == 0 && tid == 0 && a.dev_status) atomicOr(a.dev_status, TP_DEVERR_RANGE);
    }
  }
  if (e != 0.0f) c = fmaf(e1, a.entropy[t], c);
  const float nlse = -a.lse[t];
  const float2 sc2 = make_float2(a.scale, a.scale), nl2 = make_float2(nlse, nlse);
  const float2 l2e2 = make_float2(kLog2e, kLog2e);
  const float2 e2 = make_float2(e1, e1), c2 = make_float2(c, c);
  auto grad2 = [&](float x0, float x1) {
    float2 lp = __ffma2_rn(make_float2(x0, x1), sc2, nl2);
    const float2 q = __fmul2_rn(lp, l2e2);
    const float2 p = make_float2(ex2_approx(q.x), ex2_approx(q.y));
    lp = make_float2(max_nan(lp.x, kLowest), max_nan(lp.y, kLowest));
    return __fmul2_rn(p, __ffma2_rn(e2, lp, c2));
  };
  const float at_y = a.scale * g;
#pragma unroll
  for (int i = 0; i < kBwdUnits; ++i) {
    const int u = u0 + i * kBwdThreads + tid;
    if (u >= u1) break;
    const int64_t j0 = shape.head + static_cast<int64_t>(u) * kN;
    float x[kN];
    Unit<IT>::unpack(w[i], x);
#pragma unroll
    for (int q = 0; q < kN; q += 2) {
      const float2 d = grad2(x[q], x[q + 1]);
      x[q] = d.x;
      x[q + 1] = d.y;
    }
    if (y >= j0 && y < j0 + kN) {
#pragma unroll
      for (int q = 0; q < kN; ++q)
        if (j0 + q == y) x[q] += at_y;
    }
    put_unit<kN>(out + j0, x);
  }
  if (edge >= 0) put(out + edge, grad2(edge_x, 0.0f).x + (edge == y ? at_y : 0.0f));
}

// One or two tokens: the statistics of H·Eᵀ straight from one pass over E,
// which is all there is to read (2 bytes and 2·T operations a weight: CUDA
// cores keep up).  A warp takes four rows of E at once, its lanes 16-byte units
// along h; H comes from L1.  A block's 32 columns are one slice of the
// statistics that the combine below joins.  T = 1, h = 4096: v = 50304 takes 68
// us, v = 100000 127 us, 6.5 TB/s; on the tensor cores, whose tiles read the one
// row of H in every block, 93 and 155 us.  T = 3 and 4 were 88 to 95 and 159 to
// 165 us either way.
constexpr int kFewRows = 4;
constexpr int kFewPerWarp = kFewSlice / kBwdWarps;

template <int NT>
__global__ void __launch_bounds__(kBwdThreads, 4)
    linear_logprobs_few_kernel(const __nv_bfloat16* __restrict__ H,
                               const __nv_bfloat16* __restrict__ E,
                               const int64_t* __restrict__ targets, int64_t v, int h,
                               float scale, float* stat_m, float* stat_s, float* stat_u,
                               float* tgt_logit) {
  static_assert(NT <= kBwdWarps && kFewSlice % 32 == 0 && kFewPerWarp % kFewRows == 0, "");
  __shared__ float logit[NT][kFewSlice];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kFewSlice;
#pragma unroll 1
  for (int g = 0; g < kFewPerWarp; g += kFewRows) {
    const int c = warp * kFewPerWarp + g;
    const __nv_bfloat16* e[kFewRows];   // rows past the table: the last one, unused
#pragma unroll
    for (int i = 0; i < kFewRows; ++i) e[i] = E + min(col0 + c + i, v - 1) * h;
    float2 acc[kFewRows][NT];
#pragma unroll
    for (int i = 0; i < kFewRows; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[i][t] = make_float2(0.0f, 0.0f);
#pragma unroll NT == 1 ? 2 : 1
    for (int k = lane * 8; k < h; k += 256) {
      uint4 w[kFewRows];
#pragma unroll
      for (int i = 0; i < kFewRows; ++i) w[i] = ld_unit(e[i] + k);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[8];
        Unit<__nv_bfloat16>::unpack(
            __ldg(reinterpret_cast<const uint4*>(H + static_cast<int64_t>(t) * h + k)), x);
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) {
          float y[8];
          Unit<__nv_bfloat16>::unpack(w[i], y);
#pragma unroll
          for (int q = 0; q < 8; q += 2)
            acc[i][t] = __ffma2_rn(make_float2(x[q], x[q + 1]), make_float2(y[q], y[q + 1]), acc[i][t]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kFewRows; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float z = acc[i][t].x + acc[i][t].y;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
        if (lane == 0) logit[t][c + i] = z;
      }
  }
  __syncthreads();
  if (warp >= NT) return;
  // one token per warp
  constexpr int kQ = kFewSlice / 32;
  const int t = warp;
  const float sl = scale * kLog2e;
  const int64_t y = targets ? targets[t] : -1;
  float x[kQ];
  float m = -CUDART_INF_F;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int64_t col = col0 + lane + 32 * q;
    x[q] = col < v ? logit[t][lane + 32 * q] : -CUDART_INF_F;
    if (col == y) tgt_logit[t] = x[q];
    m = fmaxf(m, x[q]);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float ref = m == -CUDART_INF_F ? 0.0f : m;
  float s = 0.0f, u = 0.0f;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const float d = x[q] - ref;
    const float e = ex2_approx(d * sl);
    s += e;
    u = fmaf(e, max_nan(d, kLowest), u);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, off);
    u += __shfl_xor_sync(0xffffffffu, u, off);
  }
  if (lane == 0) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * NT + t;
    stat_m[at] = m;
    stat_s[at] = s;
    stat_u[at] = u;
  }
}

// Combine of the per-slice statistics of the output layer (slice k of
// row t at [k·T + t]): M = max m_k, w_k = exp(scale·(m_k − M)),
// S = Σ w_k·s_k, U = Σ w_k·(u_k + (m_k − M)·s_k).  A block takes eight tokens
// (a 32-byte sector of each slice's row of numbers) and 32 slices at a time, or
// one of few tokens and 256 slices; the partial results meet in a fixed order.
// One token per lane and eight slices at a time took 25 us of a T = 500,
// v = 50304 call, this takes 4.
template <int kTokens>
__global__ void __launch_bounds__(kBwdThreads)
    linear_logprobs_combine_kernel(const float* __restrict__ stat_m,
                                   const float* __restrict__ stat_s,
                                   const float* __restrict__ stat_u,
                                   const float* __restrict__ tgt_logit,
                                   const int64_t* __restrict__ targets, int64_t T, int64_t v,
                                   int nslices, float scale, float* __restrict__ logprob,
                                   float* __restrict__ entropy, float* __restrict__ lse,
                                   int32_t* dev_status) {
  constexpr int kSlices = kBwdThreads / kTokens;
  __shared__ float part_m[kBwdWarps][kTokens];
  __shared__ float part_s[kBwdWarps][kTokens];
  __shared__ float part_u[kBwdWarps][kTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = lane & (kTokens - 1);
  const int first = threadIdx.x / kTokens;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + tok;
  const bool ok = t < T;
  float m = -CUDART_INF_F;
  if (ok) {
#pragma unroll 8
    for (int k = first; k < nslices; k += kSlices) m = fmaxf(m, stat_m[k * T + t]);
  }
#pragma unroll
  for (int off = kTokens; off <= 16; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane < kTokens) part_m[warp][tok] = m;
  __syncthreads();
  float M = part_m[0][tok];
#pragma unroll
  for (int q = 1; q < kBwdWarps; ++q) M = fmaxf(M, part_m[q][tok]);
  if (M == -CUDART_INF_F) M = 0.0f;   // nothing but −inf (or NaN) in the row
  float S = 0.0f, U = 0.0f;
  if (ok) {
#pragma unroll 4
    for (int k = first; k < nslices; k += kSlices) {
      const float d = stat_m[k * T + t] - M;
      const float f = ex2_approx(d * (scale * kLog2e));
      const float s = stat_s[k * T + t];
      S = fmaf(s, f, S);
      U = fmaf(f, fmaf(fmaxf(d, kLowest), s, stat_u[k * T + t]), U);
    }
  }
#pragma unroll
  for (int off = kTokens; off <= 16; off <<= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, off);
    U += __shfl_xor_sync(0xffffffffu, U, off);
  }
  if (lane < kTokens) {
    part_s[warp][tok] = S;
    part_u[warp][tok] = U;
  }
  __syncthreads();
  if (threadIdx.x < kTokens && ok) {
    S = 0.0f;
    U = 0.0f;
#pragma unroll
    for (int q = 0; q < kBwdWarps; ++q) {
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
  // Blocks per row: one once the rows alone fill the GPU, else up to eight
  // (the portable cluster size) while each keeps a step or more of the row.
  // v = 50304, fp32: 128 rows on 1, 4, 8 blocks each take 13.9, 6.8, 8.0 us, 512
  // rows on 1, 2, 4 take 32.7, 21.4, 24.8; with 20 alternatives, whose joining
  // costs more, 16.7, 13.0, 15.6 and 29.4, 25.3, 34.7.
  const int units = static_cast<int>(a.v / Unit<IT>::kN);   // of the widest row
  const int64_t most = (kTop ? 4 : 7) * num_sms();
  int slices = 1;
  while (slices < 8 && a.T * slices * 2 <= most && units / (slices * 2) >= 2 * kThreads)
    slices *= 2;
  size_t smem = 0;
  int group_log = 0;
  if constexpr (kTop) {
    using Cand = Candidates;
    const int steps = steps_of(Part(units, 0, slices).last, kThreads * kUnits);
    group_log = group_log_of(steps, Cand::kGroups);
    smem = sizeof(Cand) + (groups_of(steps, group_log) + 3) / 4 * kThreads * sizeof(float4);
    static_assert(Cand::kGroups <= 32 && sizeof(Cand) + Cand::kGroups * kThreads * sizeof(float) <= 48 * 1024,
                  "within the default limit of dynamic shared memory");
    static_assert(Cand::kRoom >= 8 * kLogprobsMaxK, "room for the slices' best");
  }
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
  if (cudaLaunchKernelEx(&cfg, logprobs_kernel<IT, kTop>, a, slices, group_log) != cudaSuccess) {
    cudaGetLastError();
    return TP_ERR_CUDA;
  }
  note_launches(1);
  return TP_OK;
}

template <typename IT, typename GT>
tp_status logprobs_bwd_launch_t(const LogprobsBwdArgs& a, cudaStream_t stream) {
  const int64_t units = a.v / Unit<IT>::kN;
  const int64_t blocks = units > 0 ? (units + kBwdThreads * kBwdUnits - 1) / (kBwdThreads * kBwdUnits) : 1;
  if (a.T * blocks > 0x7fffffff) return TP_ERR_UNSUPPORTED;   // more logits than any GPU holds
  logprobs_bwd_kernel<IT, GT><<<static_cast<unsigned>(a.T * blocks), kBwdThreads, 0, stream>>>(
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
                                         const int64_t* targets, int64_t T, int64_t v,
                                         int nslices, float scale, float* logprob, float* entropy,
                                         float* lse, int32_t* dev_status, cudaStream_t stream) {
  auto launch = [&](auto kernel, int tokens) {
    kernel<<<static_cast<unsigned>((T + tokens - 1) / tokens), kBwdThreads, 0, stream>>>(
        stat_m, stat_s, stat_u, tgt_logit, targets, T, v, nslices, scale, logprob, entropy, lse,
        dev_status);
  };
  if (T <= kFewTokens) launch(linear_logprobs_combine_kernel<1>, 1);
  else launch(linear_logprobs_combine_kernel<8>, 8);
  note_launches(1);
  return last_error();
}

tp_status linear_logprobs_few_launch(const void* H, const void* E, const int64_t* targets,
                                     int64_t T, int64_t h, int64_t v, float scale, float* stat_m,
                                     float* stat_s, float* stat_u, float* tgt_logit,
                                     cudaStream_t stream) {
  auto launch = [&](auto kernel) {
    kernel<<<static_cast<unsigned>((v + kFewSlice - 1) / kFewSlice), kBwdThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(H), static_cast<const __nv_bfloat16*>(E), targets, v,
        static_cast<int>(h), scale, stat_m, stat_s, stat_u, tgt_logit);
  };
  static_assert(kFewTokens == 2, "one instance for each number");
  if (T == 1) launch(linear_logprobs_few_kernel<1>);
  else if (T == 2) launch(linear_logprobs_few_kernel<2>);
  else return TP_ERR_UNSUPPORTED;
  note_launches(1);
  return last_error();
}

}  // namespace tpl
