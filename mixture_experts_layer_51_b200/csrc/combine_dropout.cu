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

// Warps of a CTA sharing one token's row (1, 2, 4 or 8), a lane's first
// 8-element chunk and the stride between its chunks.
struct Place {
  int t, c0, step;
};
__device__ __forceinline__ Place place(int wpt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  return {static_cast<int>(blockIdx.x) * (kCdWarps / wpt) + warp / wpt,
          (warp % wpt) * 32 + lane, wpt * 32};
}

template <bool BF16>
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
  const int n8 = d / 8;
  uint64_t seed = 0, offset = 0;
  if (threshold) seed = rng[0], offset = rng[1];
  for (int c8 = at.c0; c8 < n8; c8 += at.step) {
    float acc[8] = {};
    for (int j = 0; j < k; ++j) {
      const int p = pos[t * k + j];
      if (p < 0) continue;
      Row8<BF16> v;
      v.load(o, p, d, c8);
      v.fma_into(gate[t * k + j], acc);
    }
    if (threshold) {
      const uint32_t keep = dropout_keep8(t * n8 + c8, offset, seed, threshold);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = (keep >> i) & 1u ? acc[i] * scale : 0.f;
    }
    if (residual) {
      Row8<BF16> r;
      r.load(residual, t, d, c8);
      r.fma_into(1.f, acc);
    }
    store8<BF16>(y, t, d, c8, acc);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kCdWarps * 32)
    combine_dropout_backward_kernel(const void* __restrict__ dy, const void* __restrict__ o,
                                    const int32_t* __restrict__ pos,
                                    const float* __restrict__ gate,
                                    const uint64_t* __restrict__ rng, uint32_t threshold,
                                    float scale, int T, int d, int k, int wpt,
                                    void* __restrict__ d_o, float* __restrict__ dgate) {
  __shared__ float part[kCdWarps][kMaxK];
  pdl_wait();
  pdl_trigger();
  const Place at = place(wpt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = at.t;
  const int n8 = d / 8;
  float dot[kMaxK] = {};
  if (at.t < T) {
    uint64_t seed = 0, offset = 0;
    if (threshold) seed = rng[0], offset = rng[1];
    for (int c8 = at.c0; c8 < n8; c8 += at.step) {
      Row8<BF16> r;
      float a[8];
      r.load(dy, t, d, c8);
      unpack8(r, a);
      uint32_t keep = 0xffu;
      if (threshold) {
        keep = dropout_keep8(t * n8 + c8, offset, seed, threshold);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = (keep >> i) & 1u ? a[i] * scale : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kMaxK; ++j) {
        const int p = j < k ? pos[t * k + j] : -1;
        if (p < 0) continue;
        float v[8];
        r.load(o, p, d, c8);
        unpack8(r, v);
        const float g = gate[t * k + j];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if ((keep >> i) & 1u) dot[j] = fmaf(a[i], v[i], dot[j]);
          v[i] = (keep >> i) & 1u ? g * a[i] : 0.f;
        }
        store8<BF16>(d_o, p, d, c8, v);
      }
    }
  }
  // The row's dot products: over the lanes, then over the warps that share it.
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
    if (lane == 0) part[warp][j] = dot[j];
  }
  __syncthreads();
  if (at.t < T && warp % wpt == 0 && lane < k) {
    float sum = 0.f;
    for (int w = 0; w < wpt; ++w) sum += part[warp + w][lane];
    dgate[t * k + lane] = pos[t * k + lane] >= 0 ? sum : 0.f;
  }
}

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
  return dtype == MOE_BF16 ? go(combine_dropout_kernel<true>) : go(combine_dropout_kernel<false>);
}

cudaError_t launch_combine_dropout_backward(const CombineDropoutArgs& a, moe_dtype dtype,
                                            cudaStream_t s) {
  const int wpt = warps_per_token(a.T, a.d), tokens = kCdWarps / wpt;
  const dim3 grid((static_cast<unsigned>(a.T) + tokens - 1) / tokens);
  auto go = [&](auto kern) {
    return launch_kernel(kern, grid, dim3(kCdWarps * 32), 0, s, 1, true, a.dy, a.o, a.pos, a.gate,
                         a.rng, a.threshold, a.scale, a.T, a.d, a.k, wpt, a.d_o, a.dgate);
  };
  return dtype == MOE_BF16 ? go(combine_dropout_backward_kernel<true>)
                           : go(combine_dropout_backward_kernel<false>);
}

}  // namespace moe
