// Declarations shared by the two halves of the router's backward pass:
// route_backward.cu (dz, the fp32 products, the sums) and
// route_backward_tc.cu (the bf16 products on the tensor cores).
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kRbTokens = 32;    // tokens of one dz block
constexpr int kRbSms = 148;      // what grids are sized for (any GPU runs them)

// dz as the tensor cores read it: bf16 terms hi + mid + lo of every value
// (24 bits in all, so the split itself costs no accuracy), side by side in
// rows of 64 * blocks elements: [hi(stride) | mid(stride) | lo(stride) | 0].
// Up to 42 experts share blocks (stride = E); above that each term has one of
// its own (stride = 64).
struct DzTerms {
  int blocks, stride;
};
inline DzTerms dz_terms(int E) {
  return E <= 21 ? DzTerms{1, E} : E <= 42 ? DzTerms{2, E} : DzTerms{3, 64};
}

// Everything a call lays out in its workspace, from the sizes alone.
struct RouteBackwardPlan {
  int EP;      // fp32: experts rounded up to 8, 16, 32 or 64; dz is [T, EP]
  int blocks;  // dz blocks
  int cols;    // column blocks of the products
  int ranges;  // token ranges of the products
  int tiles;   // token tiles, shared out over the ranges
  bool many;   // a launch of its own adds the ranges of dW_g
  size_t err, tickets, dz, bias, dw, total;  // byte offsets
};

// What the products kernels share to finish in the same launch.  `tickets`
// (one a column block, zeroed by the dz kernel of the same call) tells the
// last of a block's ranges to finish, whichever that is, to add them all up
// in order; `bias` are the dz blocks' column sums [blocks][kMaxE].
struct RouteSums {
  const float* bias;
  float* dw;          // [ranges, d, E] (three blocks of terms: [ranges, cols] parts)
  int32_t* err;
  uint32_t* tickets;
  float* dWg;         // null: not wanted
  float* dbias;
  int blocks, ranges, d, E;
  // The ranges are added by a launch of their own, and the parts are
  // [ranges, d, E] whatever the terms.
  int many;
};

// dbias of expert e by one warp: lanes over the blocks, then a tree.
__device__ __forceinline__ void sum_bias(const RouteSums& s, int e, int lane) {
  float v = 0.f;
#pragma unroll 4
  for (int b = lane; b < s.blocks; b += 32) v += s.bias[static_cast<int64_t>(b) * kMaxE + e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) s.dbias[e] = v;
}

// dW_g of columns c0 .. c0 + cols - 1: the ranges' parts in order, by `n`
// threads (this one is `i`; sync() is a barrier for all of them, scratch holds
// n pieces of 16 bytes).  One thread block reads what a whole column block
// wrote, so what counts is how many loads are on their way: eight pieces a
// thread, or, with fewer pieces than threads, several threads to a piece.
// After a time-out in the products nothing here is right: NaN says so.
template <typename Sync>
__device__ __forceinline__ void sum_ranges(const RouteSums& s, int c0, int cols, int i, int n,
                                           float4* scratch, Sync sync) {
  const int64_t plane = static_cast<int64_t>(s.d) * s.E / 4, at = static_cast<int64_t>(c0) * s.E;
  const bool failed = *static_cast<volatile int32_t*>(s.err) != 0;
  const int count = cols * s.E / 4;  // columns come in eights
  const float4* from = reinterpret_cast<const float4*>(s.dw + at);
  float4* to = reinterpret_cast<float4*>(s.dWg + at);
  auto add = [](float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; };
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float nan = __int_as_float(0x7fc00000);
  if (2 * count <= n) {
    const int groups = n / count, v = i % count, g = i / count;
    float4 sum = zero;
    if (g < groups) {
#pragma unroll 8
      for (int r = g; r < s.ranges; r += groups) add(sum, __ldcg(from + r * plane + v));
    }
    scratch[i] = sum;
    sync();
    if (i < count) {
      for (int q = 1; q < groups; ++q) add(sum, scratch[q * count + i]);
      to[i] = failed ? make_float4(nan, nan, nan, nan) : sum;
    }
    return;
  }
  constexpr int P = 8;
  for (int v0 = i; v0 < count; v0 += P * n) {
    float4 sum[P];
#pragma unroll
    for (int j = 0; j < P; ++j) sum[j] = zero;
#pragma unroll 2
    for (int r = 0; r < s.ranges; ++r) {
#pragma unroll
      for (int j = 0; j < P; ++j)
        if (v0 + j * n < count) add(sum[j], __ldcg(from + r * plane + v0 + j * n));
    }
#pragma unroll
    for (int j = 0; j < P; ++j)
      if (v0 + j * n < count) to[v0 + j * n] = failed ? make_float4(nan, nan, nan, nan) : sum[j];
  }
}

cudaError_t launch_route_products_tc(const RouteBackwardArgs& a, const RouteBackwardPlan& p,
                                     const RouteSums& sums, cudaStream_t s);
// Small batches in one launch (route_backward_small.cu).
constexpr int kRbSmallTokens = 256;
bool route_backward_is_small(int T, int d, int E);
cudaError_t launch_route_backward_small(const RouteBackwardArgs& a, moe_dtype dtype, int32_t* err,
                                        cudaStream_t s);
constexpr int kRbTcCols = 128;   // columns and tokens of one tile
constexpr int kRbTcTokens = 128;
constexpr int kRbPartBytes = 32768;  // a column block's dW_g of one range, three blocks of terms

}  // namespace moe
