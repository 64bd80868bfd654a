// The router's load-balancing loss and the per-expert counts.
//
//     counts_e = #{(t, j) : idx_tj = e},  S_e = sum_t p_te,  N = #{t}
//     L = coef E sum_e (counts_e / (N k)) (S_e / N)
//
// over the counted tokens t (all, or those the mask names).  Two launches:
// every CTA sums a slice of the tokens for all experts, then one CTA adds the
// slices in order (no floating-point atomics: the sums do not depend on
// scheduling).  Bound by reading the scores once; small batches by the
// launches.

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kBlThreads = 512;
constexpr int kBlWarps = kBlThreads / 32;
constexpr int kBlMaxSlices = 296;   // two CTAs on each of 148 SMs
constexpr int kBlMinSlice = 256;    // tokens

struct Slices {
  int n, len;  // slices, tokens in each (a multiple of 32; the last may hold fewer)
};
Slices slices(int T) {
  const int64_t per = (static_cast<int64_t>(T) + kBlMaxSlices - 1) / kBlMaxSlices;
  int64_t len = per < kBlMinSlice ? kBlMinSlice : (per + 31) / 32 * 32;
  return {static_cast<int>((T + len - 1) / len), static_cast<int>(len)};
}

// A slice's sums in the workspace: S_e, counts_e, N.
struct Partial {
  float sum[kMaxE];
  int32_t count[kMaxE];
  int32_t tokens;
  int32_t pad[3];
};

__global__ void __launch_bounds__(kBlThreads)
    balance_slice_kernel(const float* __restrict__ scores, const int32_t* __restrict__ idx,
                         const uint8_t* __restrict__ mask, int T, int E, int k, int len,
                         Partial* __restrict__ out) {
  __shared__ int32_t cnt[kMaxE];
  __shared__ int32_t ntok;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blockIdx.x * len, t1 = min(T, t0 + len);
  if (tid < kMaxE) cnt[tid] = 0;
  if (tid == 0) ntok = 0;
  __syncthreads();
  for (int t = t0 + tid; t < t1; t += kBlThreads) {
    if (mask && !mask[t]) continue;
    atomicAdd(&ntok, 1);
    for (int j = 0; j < k; ++j) {
      const int e = idx[static_cast<int64_t>(t) * k + j];
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
  }
  Partial& p = out[blockIdx.x];
  for (int e = warp; e < E; e += kBlWarps) {
    float s = 0.f;
    for (int t = t0 + lane; t < t1; t += 32)
      if (!mask || mask[t]) s += scores[static_cast<int64_t>(e) * T + t];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) p.sum[e] = s;
  }
  __syncthreads();
  if (tid < E) p.count[tid] = cnt[tid];
  if (tid == 0) p.tokens = ntok;
}

__global__ void __launch_bounds__(kMaxE)
    balance_finish_kernel(const Partial* __restrict__ part, int n, int E, int k, float coef,
                          float* __restrict__ loss, float* __restrict__ prob_sum,
                          int32_t* __restrict__ counts, int32_t* __restrict__ tokens) {
  __shared__ double term[kMaxE];
  pdl_wait();
  pdl_trigger();
  const int e = threadIdx.x;
  float sum = 0.f;
  int32_t count = 0, tok = 0;
  for (int s = 0; s < n; ++s) {
    if (e < E) {
      sum += part[s].sum[e];
      count += part[s].count[e];
    }
    tok += part[s].tokens;
  }
  if (e < E) {
    prob_sum[e] = sum;
    counts[e] = count;
  }
  term[e] = e < E && tok > 0 ? static_cast<double>(count) / k * sum / tok / tok : 0.0;
  __syncthreads();
  if (e == 0) {
    double total = 0.0;
    for (int i = 0; i < E; ++i) total += term[i];
    *loss = static_cast<float>(coef * E * total);
    *tokens = tok;
  }
}

}  // namespace

size_t balance_scratch_bytes(int T) { return sizeof(Partial) * (slices(T).n + 1); }

cudaError_t launch_balance_loss(const BalanceArgs& a, cudaStream_t s) {
  const Slices sl = slices(a.T);
  Partial* part = static_cast<Partial*>(a.ws);
  if (sl.n > 0) {
    const cudaError_t err =
        launch_kernel(balance_slice_kernel, dim3(sl.n), dim3(kBlThreads), 0, s, 1, true, a.scores,
                      a.idx, a.mask, a.T, a.E, a.k, sl.len, part);
    if (err != cudaSuccess) return err;
  }
  return launch_kernel(balance_finish_kernel, dim3(1), dim3(kMaxE), 0, s, 1, true,
                       static_cast<const Partial*>(part), sl.n, a.E, a.k, a.coef, a.loss,
                       a.prob_sum, a.counts, a.tokens);
}

}  // namespace moe
