// The router's load-balancing loss and the per-expert counts.
//
//     counts_e = #{(t, j) : idx_tj = e},  S_e = sum_t p_te,  N = #{t}
//     L = coef E sum_e (counts_e / (N k)) (S_e / N)
//
// over the counted tokens t (all, or those the mask names).  Every CTA sums a
// slice of the tokens for all experts; the slices are added in order (no
// floating-point atomics: the sums do not depend on scheduling).
//
// Bound by reading the scores once, and for small batches by launches and
// round trips to memory.  So a batch of up to 64 KB (scores and indices) is
// one CTA's, one of up to 768 KB a cluster's of eight CTAs, whose first adds
// the others' sums out of their shared memory, and a larger one takes a CTA on
// every SM and a second launch that adds the slices from the workspace.
//
// Measured back to back in a graph on one B200 (with eight scores a lane on
// their way, which costs small batches 0.5 us and large ones nothing): 5 KB
// 3.9 us in one CTA, 4.8 as a cluster; 147 KB 5.4 and 4.9; 590 KB 4.9 as a
// cluster, 5.7 in two launches; 1.2 MB 6.4 and 5.7.  As built: 256 tokens of 4
// experts 3.3 us, 8192 of 8 5.1 us, 100003 of 64 with a mask (29 MB) 9.0 us;
// reading that takes 4.4 us at 6.56 TB/s, the rest is two launches and the
// last sums.  The mask as one word of ballots for 32 tokens, instead of a byte
// beside every score: 12.1 -> 8.7 us.

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
static_assert(kWarps == 32, "a warp adds up the warps");
constexpr int kCluster = 8;
constexpr int64_t kOneBytes = 1 << 16;      // scores and indices that one CTA takes,
constexpr int64_t kClusterBytes = 3 << 18;  // and one cluster
constexpr int kMaxSlices = 148;     // one CTA on each SM
constexpr int kMinSlice = 256;      // tokens
constexpr int kBatch = 4;           // scores a lane has on their way per expert

// A slice's sums: S_e, counts_e, N.
struct Partial {
  float sum[kMaxE];
  int32_t count[kMaxE];
  int32_t tokens;
  int32_t pad[3];
};

struct Slices {
  int n, len;  // slices, tokens in each (a multiple of 32; the last may hold fewer)
};
Slices slices(int T) {
  const int64_t per = (static_cast<int64_t>(T) + kMaxSlices - 1) / kMaxSlices;
  const int64_t len = per < kMinSlice ? kMinSlice : (per + 31) / 32 * 32;
  return {static_cast<int>((T + len - 1) / len), static_cast<int>(len)};
}

// The sums over tokens t0 .. t1 - 1 into `out` (shared memory), by the whole
// CTA, 1024 tokens at a time: thread i asks for its token's mask and experts,
// a warp for an expert's scores, 32 kBatch tokens at a time (with fewer than
// 32 experts several warps share one, each with a part of the tokens).
__device__ void sum_slice(const float* __restrict__ scores, const int32_t* __restrict__ idx,
                          const uint8_t* __restrict__ mask, int T, int E, int k, uint32_t t0,
                          uint32_t t1, Partial& out) {
  __shared__ float part[kWarps][2];  // a warp's experts: at most two
  __shared__ int32_t count_s[kMaxE];
  __shared__ uint32_t on_s[kWarps];  // bit l of word w: token 32 w + l counts
  __shared__ int32_t tokens_s[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kMaxE) count_s[tid] = 0;
  // Experts of a round of warps (a power of two), and warps to an expert.
  const int wide = E > 16 ? 32 : E > 8 ? 16 : E > 4 ? 8 : E > 2 ? 4 : E;
  const int share = kWarps / wide, e0 = warp % wide, q = warp / wide;
  float s[2] = {0.f, 0.f};
  int32_t tokens = 0;
  for (uint32_t c0 = t0; c0 < t1; c0 += kThreads) {
    const uint32_t c1 = t1 - c0 < kThreads ? t1 : c0 + kThreads, tok = c0 + tid;
    const bool counted = tok < c1 && (!mask || mask[tok]);
    int sel[kMaxK];
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      sel[j] = tok < c1 && j < k ? __ldg(idx + static_cast<int64_t>(tok) * k + j) : -1;
    bool first = true;
    for (uint32_t t = c0 + q * 32 * kBatch; t < c1 || first; t += share * 32 * kBatch) {
      float v[2][kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t at = t + 32 * i + lane;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = e0 + h * wide;
          v[h][i] = at < c1 && e < E ? __ldg(scores + static_cast<int64_t>(e) * T + at) : 0.f;
        }
      }
      if (first) {
        // Every load of the first batch is on its way: now the mask's words.
        const unsigned word = __ballot_sync(0xffffffffu, counted);
        if (lane == 0) on_s[warp] = word;
        tokens += __popc(word);
        first = false;
        __syncthreads();
      }
      // A token that does not count may hold anything: left out, not times 0.
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t w = (t - c0) / 32 + i;
        const bool on = w < kWarps && (on_s[w % kWarps] >> lane & 1u);
#pragma unroll
        for (int h = 0; h < 2; ++h) s[h] += on ? v[h][i] : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (counted && sel[j] >= 0 && sel[j] < E) atomicAdd(&count_s[sel[j]], 1);
    if (t1 - c0 > kThreads) __syncthreads();  // before the next words
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s[h] += __shfl_xor_sync(0xffffffffu, s[h], o);
    if (lane == 0) part[warp][h] = s[h];
  }
  if (lane == 0) tokens_s[warp] = tokens;
  __syncthreads();
  if (tid < kMaxE) {
    float total = 0.f;
    if (tid < E)
      for (int i = 0; i < share; ++i) total += part[tid % wide + i * wide][tid / wide];
    out.sum[tid] = total;
    out.count[tid] = count_s[tid];
  } else if (warp == kMaxE / 32) {
    int32_t n = tokens_s[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) out.tokens = n;
  }
}

// The loss from the totals, by the first two warps (thread e: expert e).
__device__ __forceinline__ void finish(int e, int E, int k, float coef, float sum, int32_t count,
                                       int32_t tokens, const BalanceArgs& a) {
  __shared__ double half;
  double term = 0.0;
  if (e < E) {
    a.prob_sum[e] = sum;
    a.counts[e] = count;
    if (tokens > 0) term = static_cast<double>(count) / k * sum / tokens / tokens;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
  if (e == 32) half = term;
  asm volatile("bar.sync 1, 64;" ::: "memory");
  if (e == 0) {
    *a.loss = static_cast<float>(coef * E * (term + half));
    *a.tokens = tokens;
  }
}

// C CTAs of one cluster.
template <int C>
__global__ void __launch_bounds__(kThreads, 1) balance_cluster_kernel(const BalanceArgs a, int len) {
  __shared__ Partial mine;
  const int tid = threadIdx.x;
  const uint32_t rank = C > 1 ? cluster_ctarank() : 0;
  pdl_wait();
  pdl_trigger();
  const int t0 = min(a.T, static_cast<int>(rank) * len), t1 = min(a.T, t0 + len);
  sum_slice(a.scores, a.idx, a.mask, a.T, a.E, a.k, t0, t1, mine);
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  if (rank == 0 && tid < kMaxE) {
    float sum = 0.f;
    int32_t count = 0, tokens = 0;
    uint32_t v[C][3];
#pragma unroll
    for (int r = 0; r < C; ++r) {
      const uint32_t from = mapa_shared(smem_u32(&mine), r);
      v[r][0] = ld_shared_cluster_u32(from + offsetof(Partial, sum) + 4 * tid);
      v[r][1] = ld_shared_cluster_u32(from + offsetof(Partial, count) + 4 * tid);
      v[r][2] = ld_shared_cluster_u32(from + offsetof(Partial, tokens));
    }
#pragma unroll
    for (int r = 0; r < C; ++r) {
      sum += __uint_as_float(v[r][0]);
      count += static_cast<int32_t>(v[r][1]);
      tokens += static_cast<int32_t>(v[r][2]);
    }
    finish(tid, a.E, a.k, a.coef, sum, count, tokens, a);
  }
  if (C > 1) cluster_sync();  // the others' shared memory lives until it has been read
}

__global__ void __launch_bounds__(kThreads, 1) balance_slice_kernel(const BalanceArgs a, int len) {
  __shared__ Partial mine;
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * len, t1 = a.T - t0 < len ? a.T : t0 + len;
  sum_slice(a.scores, a.idx, a.mask, a.T, a.E, a.k, t0, t1, mine);
  __syncthreads();
  const uint32_t* from = reinterpret_cast<const uint32_t*>(&mine);
  uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<Partial*>(a.ws) + blockIdx.x);
  for (int i = threadIdx.x; i < static_cast<int>(offsetof(Partial, pad)) / 4; i += kThreads)
    to[i] = from[i];
}

__global__ void __launch_bounds__(kThreads, 1) balance_finish_kernel(const BalanceArgs a, int n) {
  constexpr int G = kThreads / kMaxE;  // threads to an expert
  __shared__ float sum_s[G][kMaxE];
  __shared__ int32_t count_s[G][kMaxE], tokens_s[G];
  pdl_wait();
  pdl_trigger();
  const int e = threadIdx.x % kMaxE, g = threadIdx.x / kMaxE;
  const Partial* part = static_cast<const Partial*>(a.ws);
  constexpr int R = (kMaxSlices + G - 1) / G;  // slices a thread adds, all on their way at once
  float sums[R];
  int32_t counts[R], toks[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int s = g + i * G;
    sums[i] = s < n ? part[s].sum[e] : 0.f;
    counts[i] = s < n ? part[s].count[e] : 0;
    toks[i] = s < n && e == 0 ? part[s].tokens : 0;
  }
  float sum = 0.f;
  int32_t count = 0, tokens = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) sum += sums[i], count += counts[i], tokens += toks[i];
  sum_s[g][e] = sum;
  count_s[g][e] = count;
  if (e == 0) tokens_s[g] = tokens;
  __syncthreads();
  if (g > 0) return;
  tokens = tokens_s[0];
#pragma unroll
  for (int i = 1; i < G; ++i) {
    sum += sum_s[i][e];
    count += count_s[i][e];
    tokens += tokens_s[i];
  }
  finish(e, a.E, a.k, a.coef, sum, count, tokens, a);
}

}  // namespace

size_t balance_scratch_bytes(int T) { return sizeof(Partial) * (slices(T).n + 1); }

cudaError_t launch_balance_loss(const BalanceArgs& a, cudaStream_t s) {
  const int64_t bytes = static_cast<int64_t>(a.T) * (a.E + a.k) * 4;
  if (bytes <= kOneBytes)
    return launch_kernel(balance_cluster_kernel<1>, dim3(1), dim3(kThreads), 0, s, 1, true, a, a.T);
  if (bytes <= kClusterBytes)
    return launch_kernel(balance_cluster_kernel<kCluster>, dim3(kCluster), dim3(kThreads), 0, s,
                         kCluster, true, a, (a.T + 32 * kCluster - 1) / (32 * kCluster) * 32);
  const Slices sl = slices(a.T);
  const cudaError_t err = launch_kernel(balance_slice_kernel, dim3(sl.n), dim3(kThreads), 0, s, 1,
                                        true, a, sl.len);
  if (err != cudaSuccess) return err;
  return launch_kernel(balance_finish_kernel, dim3(1), dim3(kThreads), 0, s, 1, true, a, sl.n);
}

}  // namespace moe
