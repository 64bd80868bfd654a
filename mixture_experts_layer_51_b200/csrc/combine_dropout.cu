// Un-permute and gate-weighted combine with dropout and the residual, and its
// backward pass:
//
//     y_tc  = r_tc + m_tc sum_j g_tj o[pos_tj, c]
//     d_o[pos_tj, c] = g_tj a_tc,   d_g_tj = sum_c a_tc o[pos_tj, c],
//     a_tc = m_tc dy_tc
//
// with m_tc = 0 for a dropped element and 1 / (1 - p) for the others, made
// afresh from the generator of philox.cuh in both directions: the mask is
// never stored.  A dropped element is left out, not multiplied by zero, so
// what stands there (infinities, NaN) reaches neither y nor a gradient.
//
// One token's row is owned by whole warps of one CTA, so the k gate gradients
// are a fixed-order sum and nothing is atomic; every permuted row belongs to
// one (token, slot), so the scatter of d_o writes each row once.

#include "moe_internal.cuh"
#include "philox.cuh"

namespace moe {
namespace {

constexpr int kCdWarps = 8;

__device__ __forceinline__ void unpack8(const Row8<true>& r, float (&f)[8]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Row8<false>& r, float (&f)[8]) {
  f[0] = r.a.x, f[1] = r.a.y, f[2] = r.a.z, f[3] = r.a.w;
  f[4] = r.b.x, f[5] = r.b.y, f[6] = r.b.z, f[7] = r.b.w;
}

template <bool BF16>
__device__ __forceinline__ void store8(void* y, int64_t row, int d, int c8, const float (&v)[8]) {
  if (BF16) {
    uint4 q;
    q.x = pack_bf16x2(v[0], v[1]);
    q.y = pack_bf16x2(v[2], v[3]);
    q.z = pack_bf16x2(v[4], v[5]);
    q.w = pack_bf16x2(v[6], v[7]);
    reinterpret_cast<uint4*>(y)[row * (d / 8) + c8] = q;
  } else {
    float4* r = reinterpret_cast<float4*>(y) + row * (d / 4) + c8 * 2;
    r[0] = make_float4(v[0], v[1], v[2], v[3]);
    r[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Warps of a CTA sharing one token's row (1, 2, 4 or 8): this warp's token,
// and which of the token's warps it is.
struct Place {
  int t, part;
};
__device__ __forceinline__ Place place(int wpt) {
  const int warp = threadIdx.x >> 5;
  return {static_cast<int>(blockIdx.x) * (kCdWarps / wpt) + warp / wpt, warp % wpt};
}

// The token's rows and gates, in every lane (row -1: no such slot).
template <int KJ>
__device__ __forceinline__ void slots(const int32_t* pos, const float* gate, int64_t t, int k,
                                      int (&row)[KJ], float (&g)[KJ]) {
  const int lane = threadIdx.x & 31;
  const int pl = lane < k ? pos[t * k + lane] : -1;
  const float gl = lane < k ? gate[t * k + lane] : 0.f;
#pragma unroll
  for (int j = 0; j < KJ; ++j) {
    row[j] = __shfl_sync(0xffffffffu, pl, j);
    g[j] = __shfl_sync(0xffffffffu, gl, j);
  }
}

// KJ = slots this instantiation handles (2 for k <= 2, else kMaxK); CH =
// 8-element chunks of each row per lane and iteration: every load of an
// iteration is issued before any arithmetic (the generator's, too, runs while
// they are on their way).
template <bool BF16, int KJ, int CH>
__global__ void __launch_bounds__(kCdWarps * 32)
    combine_dropout_kernel(const void* __restrict__ o, const int32_t* __restrict__ pos,
                           const float* __restrict__ gate, const void* residual,
                           const uint64_t* __restrict__ rng, uint32_t threshold, float scale,
                           int T, int d, int k, int wpt, void* y) {
  pdl_wait();
  pdl_trigger();
  const Place at = place(wpt);
  if (at.t >= T) return;
  const int64_t t = at.t;
  const int n8 = d / 8, lane = threadIdx.x & 31;
  uint64_t seed = 0, offset = 0;
  if (threshold) seed = rng[0], offset = rng[1];
  int row[KJ];
  float g[KJ];
  slots<KJ>(pos, gate, t, k, row, g);
  for (int c0 = at.part * 32 * CH + lane; c0 < n8; c0 += wpt * 32 * CH) {
    Row8<BF16> v[KJ][CH], res[CH];
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      const int c8 = c0 + h * 32;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        if (row[j] >= 0 && c8 < n8)
          v[j][h].load(o, row[j], d, c8);
        else
          v[j][h].zero();
      }
      if (residual && c8 < n8)
        res[h].load(residual, t, d, c8);
      else
        res[h].zero();
    }
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      const int c8 = c0 + h * 32;
      if (c8 >= n8) break;
      uint32_t w[4];
      if (threshold) philox4x32_10(t * n8 + c8, offset, seed, w);
      float acc[8] = {};
#pragma unroll
      for (int j = 0; j < KJ; ++j)
        if (row[j] >= 0) v[j][h].fma_into(g[j], acc);  // absent slots add nothing
      if (threshold) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = dropout_kept(w, i, threshold) ? acc[i] * scale : 0.f;
      }
      if (residual) res[h].fma_into(1.f, acc);
      store8<BF16>(y, t, d, c8, acc);
    }
  }
}

// Adds `v` over the 32 lanes: afterwards lane l holds in the result the total
// of v[l / (32 / N) % N], each added in an order that is always the same.
template <int N>
__device__ __forceinline__ float reduce_lanes(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int s = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, s /= 2) {
    // The upper half of the lanes keeps the upper half of the values.
    const bool upper = lane & s;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = upper ? v[i] : v[i + n];
      const float keep = upper ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
    }
  }
#pragma unroll
  for (; s > 0; s /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
  return v[0];
}

template <bool BF16, int KJ, int CH>
__global__ void __launch_bounds__(kCdWarps * 32)
    combine_dropout_backward_kernel(const void* __restrict__ dy, const void* __restrict__ o,
                                    const int32_t* __restrict__ pos,
                                    const float* __restrict__ gate,
                                    const uint64_t* __restrict__ rng, uint32_t threshold,
                                    float scale, int T, int d, int k, int wpt,
                                    void* __restrict__ d_o, float* __restrict__ dgate) {
  __shared__ float part[kCdWarps][KJ];
  pdl_wait();
  pdl_trigger();
  const Place at = place(wpt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = at.t;
  const int n8 = d / 8;
  float dot[KJ] = {};
  int row[KJ];
#pragma unroll
  for (int j = 0; j < KJ; ++j) row[j] = -1;
  if (at.t < T) {
    float g[KJ];
    uint64_t seed = 0, offset = 0;
    if (threshold) seed = rng[0], offset = rng[1];
    slots<KJ>(pos, gate, t, k, row, g);
#pragma unroll
    for (int j = 0; j < KJ; ++j) g[j] *= scale;
    for (int c0 = at.part * 32 * CH + lane; c0 < n8; c0 += wpt * 32 * CH) {
      Row8<BF16> v[KJ][CH], up[CH];
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        const int c8 = c0 + h * 32;
        if (c8 >= n8) break;
        up[h].load(dy, t, d, c8);
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          if (row[j] >= 0) v[j][h].load(o, row[j], d, c8);
      }
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        const int c8 = c0 + h * 32;
        if (c8 >= n8) break;
        // Dropped elements become zero in dy and in o (what o holds there is
        // left out: 0 times it need not be 0), halfword masks for both.
        uint32_t m[4];
        if (threshold) {
          philox4x32_10(t * n8 + c8, offset, seed, m);
#pragma unroll
          for (int i = 0; i < 4; ++i) m[i] = __vcmpgeu2(m[i], threshold << 16 | threshold);
          up[h].mask(m);
        }
        float a[8];
        unpack8(up[h], a);
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          if (row[j] < 0) continue;
          if (threshold) v[j][h].mask(m);
          float f[8];
          unpack8(v[j][h], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(a[i], f[i], dot[j]);
            f[i] = g[j] * a[i];  // g carries the scale
          }
          store8<BF16>(d_o, row[j], d, c8, f);
        }
      }
    }
  }
  // The row's dot products: over the lanes, then over the warps that share it.
  const float sum = scale * reduce_lanes<KJ>(dot);
  constexpr int W = 32 / KJ;  // lanes that hold the same total
  if (wpt == 1) {
    if (at.t < T && lane % W == 0 && lane / W < k)
      dgate[t * k + lane / W] = pos[t * k + lane / W] >= 0 ? sum : 0.f;
    return;
  }
  if (lane % W == 0) part[warp][lane / W] = sum;
  __syncthreads();
  if (at.t < T && at.part == 0 && lane < k) {
    float total = 0.f;
    for (int i = 0; i < wpt; ++i) total += part[warp + i][lane];
    dgate[t * k + lane] = pos[t * k + lane] >= 0 ? total : 0.f;
  }
}

// Warps a token: one where the tokens alone fill the GPU (eight warps on each
// of 148 SMs), else as many as it takes, while each keeps a whole sweep of a
// row (256 elements) to itself.
int warps_per_token(int T, int d) {
  int wpt = 1;
  while (wpt < kCdWarps && static_cast<int64_t>(T) * wpt < 148 * kCdWarps && wpt * 256 < d) wpt *= 2;
  return wpt;
}

}  // namespace

cudaError_t launch_combine_dropout(const CombineDropoutArgs& a, moe_dtype dtype, cudaStream_t s) {
  const int wpt = warps_per_token(a.T, a.d), tokens = kCdWarps / wpt;
  const dim3 grid((static_cast<unsigned>(a.T) + tokens - 1) / tokens);
  auto go = [&](auto kern) {
    return launch_kernel(kern, grid, dim3(kCdWarps * 32), 0, s, 1, true, a.o, a.pos, a.gate,
                         a.residual, a.rng, a.threshold, a.scale, a.T, a.d, a.k, wpt, a.y);
  };
  if (dtype == MOE_BF16)
    return a.k <= 2 ? go(combine_dropout_kernel<true, 2, 4>)
                    : go(combine_dropout_kernel<true, kMaxK, 2>);
  return a.k <= 2 ? go(combine_dropout_kernel<false, 2, 2>)
                  : go(combine_dropout_kernel<false, kMaxK, 1>);
}

cudaError_t launch_combine_dropout_backward(const CombineDropoutArgs& a, moe_dtype dtype,
                                            cudaStream_t s) {
  const int wpt = warps_per_token(a.T, a.d), tokens = kCdWarps / wpt;
  const dim3 grid((static_cast<unsigned>(a.T) + tokens - 1) / tokens);
  auto go = [&](auto kern) {
    return launch_kernel(kern, grid, dim3(kCdWarps * 32), 0, s, 1, true, a.dy, a.o, a.pos, a.gate,
                         a.rng, a.threshold, a.scale, a.T, a.d, a.k, wpt, a.d_o, a.dgate);
  };
  if (dtype == MOE_BF16)
    return a.k <= 2 ? go(combine_dropout_backward_kernel<true, 2, 2>)
                    : go(combine_dropout_backward_kernel<true, kMaxK, 1>);
  return a.k <= 2 ? go(combine_dropout_backward_kernel<false, 2, 1>)
                  : go(combine_dropout_backward_kernel<false, kMaxK, 1>);
}

}  // namespace moe
