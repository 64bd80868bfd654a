// Backward pass of the router: from the gradients of the gates and of the
// balance loss to the gradients of x, W_g and the bias.
//
// With p = softmax over all experts (scores), g the gates, s the gate scale,
// f_e = counts_e / (N k) the share of the assignments that expert e got:
//
//   TopK, then softmax:  dz_{idx_j} += g_j (dg_j - sum_i (g_i / s) dg_i)
//   softmax, then TopK:  dz_e += [e = idx_j] g_j dg_j - p_e sum_i g_i dg_i
//   balance loss:        dz_e += dL coef (E / N) p_e (f_e - sum_i f_i p_i)
//   dx = dx_acc + dz W_g^T,   dW_g = x^T dz,   dbias = sum_t dz
//
// Three launches.  (1) dz for every token, and its column sums per block of
// tokens.  (2) Both products in one pass over x: a CTA owns a block of
// columns and a range of tokens, so each x element is read once, each dx
// element written once, and dW_g of the block stays on the chip until the
// range is done.  (3) The ranges' dW_g and the blocks' column sums added in
// order (no floating-point atomics).

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kRbTokens = 128;    // tokens of one dz block
constexpr int kRbCols = 64;       // columns of one product CTA
constexpr int kRbTile = 32;       // tokens of one tile
constexpr int kRbThreads = 256;

// Experts rounded up to the widths the product kernels are built for.
int padded_experts(int E) { return E <= 8 ? 8 : E <= 16 ? 16 : E <= 32 ? 32 : 64; }

struct Plan {
  int EP;           // padded experts: dz is [T, EP], zero past E
  int blocks;       // dz blocks
  int cols;         // column blocks
  int ranges;       // token ranges
  int range;        // tokens of a range (a multiple of kRbTile)
  size_t dz, bias, dw, total;  // byte offsets in the workspace
};

Plan make_plan(int T, int d, int E) {
  Plan p;
  p.EP = padded_experts(E);
  p.blocks = (T + kRbTokens - 1) / kRbTokens;
  p.cols = (d + kRbCols - 1) / kRbCols;
  const int tiles = (T + kRbTile - 1) / kRbTile;
  int want = (148 * 4 + p.cols - 1) / p.cols;
  if (want > tiles) want = tiles;
  if (want < 1) want = 1;
  p.range = (tiles + want - 1) / want * kRbTile;
  p.ranges = p.range ? (T + p.range - 1) / p.range : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  p.dz = take(sizeof(float) * p.EP * static_cast<size_t>(T));
  p.bias = take(sizeof(float) * kMaxE * static_cast<size_t>(p.blocks));
  p.dw = take(sizeof(float) * d * static_cast<size_t>(E) * p.ranges);
  p.total = at;
  return p;
}

// One thread a token: its row of dz, through shared memory so that the block
// writes whole rows, and the block's column sums.
__global__ void __launch_bounds__(kRbTokens)
    route_dz_kernel(RouteBackwardArgs a, int EP, float* __restrict__ dz,
                    float* __restrict__ bias_part) {
  extern __shared__ float row_s[];  // [EP][kRbTokens]
  __shared__ float f[kMaxE];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int t = blockIdx.x * kRbTokens + tid;
  float c = 0.f;
  if (a.counts) {
    const int n = *a.tokens;
    if (n > 0) {
      c = a.coef * (a.dloss ? *a.dloss : 1.f) * a.E / n;
      if (tid < a.E) f[tid] = static_cast<float>(a.counts[tid]) / (static_cast<float>(n) * a.k);
    } else if (tid < a.E) {
      f[tid] = 0.f;
    }
  }
  for (int e = 0; e < EP; ++e) row_s[e * kRbTokens + tid] = 0.f;
  __syncthreads();
  if (t < a.T && (!a.mask || a.mask[t])) {
    float total = 0.f, mean = 0.f;
    if (a.dgate)
      for (int j = 0; j < a.k; ++j)
        total = fmaf(a.gate[static_cast<int64_t>(t) * a.k + j],
                     a.dgate[static_cast<int64_t>(t) * a.k + j], total);
    if (a.counts)
      for (int e = 0; e < a.E; ++e)
        mean = fmaf(f[e], a.scores[static_cast<int64_t>(e) * a.T + t], mean);
    const bool all = a.dgate && a.gating == MOE_GATE_SOFTMAX_TOPK;
    if (a.counts || all)
      for (int e = 0; e < a.E; ++e) {
        const float p = a.scores[static_cast<int64_t>(e) * a.T + t];
        row_s[e * kRbTokens + tid] = (a.counts ? c * p * (f[e] - mean) : 0.f) - (all ? p * total : 0.f);
      }
    if (a.dgate)
      for (int j = 0; j < a.k; ++j) {
        const int e = a.idx[static_cast<int64_t>(t) * a.k + j];
        if (e < 0 || e >= a.E) continue;
        const float g = a.gate[static_cast<int64_t>(t) * a.k + j];
        const float dg = a.dgate[static_cast<int64_t>(t) * a.k + j];
        row_s[e * kRbTokens + tid] += all ? g * dg : g * (dg - total / a.gate_scale);
      }
  }
  __syncthreads();
  const int rows = min(kRbTokens, a.T - static_cast<int>(blockIdx.x) * kRbTokens);
  float* out = dz + static_cast<int64_t>(blockIdx.x) * kRbTokens * EP;
  for (int i = tid; i < rows * EP; i += kRbTokens) out[i] = row_s[(i % EP) * kRbTokens + i / EP];
  if (tid < a.E) {
    float s = 0.f;
    for (int i = 0; i < rows; ++i) s += row_s[tid * kRbTokens + i];
    bias_part[static_cast<int64_t>(blockIdx.x) * kMaxE + tid] = s;
  }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  return reinterpret_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16(v);
  else
    reinterpret_cast<float*>(p)[i] = v;
}

// Both products on fp32 FMA: thread (column, quarter) keeps its column's
// share of dW_g (a quarter of the experts) and its column of W_g in
// registers, and makes dx for a quarter of the tile's tokens.
template <bool BF16, int EP>
__global__ void __launch_bounds__(kRbThreads)
    route_products_kernel(RouteBackwardArgs a, int range, const float* __restrict__ dz,
                          float* __restrict__ dw) {
  constexpr int QE = EP / 4;
  __shared__ __align__(16) float dz_s[kRbTile][EP];
  __shared__ float x_s[kRbTile][kRbCols];
  const int tid = threadIdx.x, col = tid % kRbCols, q = tid / kRbCols;
  const int c = blockIdx.x * kRbCols + col;
  const bool in = c < a.d;
  pdl_wait();
  pdl_trigger();
  float w[EP], acc[QE];
#pragma unroll
  for (int e = 0; e < EP; ++e)
    w[e] = a.dx && in && e < a.E ? load1<BF16>(a.Wg, static_cast<int64_t>(c) * a.E + e) : 0.f;
#pragma unroll
  for (int e = 0; e < QE; ++e) acc[e] = 0.f;
  const int t0 = blockIdx.y * range, t1 = min(a.T, t0 + range);
  for (int tb = t0; tb < t1; tb += kRbTile) {
    __syncthreads();
    const int rows = min(kRbTile, t1 - tb);
    for (int i = tid; i < kRbTile * EP; i += kRbThreads)
      (&dz_s[0][0])[i] = i < rows * EP ? dz[static_cast<int64_t>(tb) * EP + i] : 0.f;
    if (a.dWg)
      for (int r = q; r < kRbTile; r += 4) {
        const int t = tb + r;
        const bool use = in && r < rows && (!a.mask || a.mask[t]);
        x_s[r][col] = use ? load1<BF16>(a.x, static_cast<int64_t>(t) * a.d + c) : 0.f;
      }
    __syncthreads();
    if (a.dWg)
      for (int r = 0; r < kRbTile; ++r) {
        const float xv = x_s[r][col];
#pragma unroll
        for (int e = 0; e < QE; ++e) acc[e] = fmaf(xv, dz_s[r][q * QE + e], acc[e]);
      }
    if (a.dx && in)
      for (int r = q; r < rows; r += 4) {
        const int64_t at = static_cast<int64_t>(tb + r) * a.d + c;
        float v = 0.f;
#pragma unroll
        for (int e = 0; e < EP; ++e) v = fmaf(dz_s[r][e], w[e], v);
        if (a.dx_acc) v += load1<BF16>(a.dx_acc, at);
        store1<BF16>(a.dx, at, v);
      }
  }
  if (a.dWg && in)
#pragma unroll
    for (int e = 0; e < QE; ++e)
      if (q * QE + e < a.E)
        dw[(static_cast<int64_t>(blockIdx.y) * a.d + c) * a.E + q * QE + e] = acc[e];
}

__global__ void __launch_bounds__(256)
    route_finish_kernel(const float* __restrict__ dw, const float* __restrict__ bias_part,
                        int ranges, int blocks, int64_t n, int E, float* __restrict__ dWg,
                        float* __restrict__ dbias) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (dWg && i < n) {
    float s = 0.f;
    for (int r = 0; r < ranges; ++r) s += dw[r * n + i];
    dWg[i] = s;
  }
  if (dbias && i < E) {
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += bias_part[static_cast<int64_t>(b) * kMaxE + i];
    dbias[i] = s;
  }
}

template <bool BF16>
cudaError_t launch_products(const RouteBackwardArgs& a, const Plan& p, const float* dz, float* dw,
                            cudaStream_t s) {
  auto go = [&](auto kern) {
    return launch_kernel(kern, dim3(p.cols, p.ranges), dim3(kRbThreads), 0, s, 1, true, a, p.range,
                         dz, dw);
  };
  switch (p.EP) {
    case 8: return go(route_products_kernel<BF16, 8>);
    case 16: return go(route_products_kernel<BF16, 16>);
    case 32: return go(route_products_kernel<BF16, 32>);
    default: return go(route_products_kernel<BF16, 64>);
  }
}

}  // namespace

size_t route_backward_scratch_bytes(int T, int d, int E, moe_dtype) {
  return make_plan(T, d, E).total;
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, moe_dtype dtype, cudaStream_t s) {
  const Plan p = make_plan(a.T, a.d, a.E);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  float* dz = reinterpret_cast<float*>(ws + p.dz);
  float* bias_part = reinterpret_cast<float*>(ws + p.bias);
  float* dw = reinterpret_cast<float*>(ws + p.dw);
  cudaError_t err = cudaSuccess;
  if (a.T > 0) {
    err = launch_kernel(route_dz_kernel, dim3(p.blocks), dim3(kRbTokens),
                        sizeof(float) * p.EP * kRbTokens, s, 1, true, a, p.EP, dz, bias_part);
    if (err == cudaSuccess && (a.dx || a.dWg))
      err = dtype == MOE_BF16 ? launch_products<true>(a, p, dz, dw, s)
                              : launch_products<false>(a, p, dz, dw, s);
    if (err != cudaSuccess) return err;
  }
  if (!a.dWg && !a.dbias) return cudaSuccess;
  const int64_t n = static_cast<int64_t>(a.d) * a.E;
  return launch_kernel(route_finish_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256),
                       0, s, 1, true, static_cast<const float*>(dw),
                       static_cast<const float*>(bias_part), p.ranges, p.blocks, n, a.E, a.dWg,
                       a.dbias);
}

}  // namespace moe
