// Declarations shared by the two halves of the router's backward pass:
// route_backward.cu (dz, the fp32 products, the sums) and
// route_backward_tc.cu (the bf16 products on the tensor cores).
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kRbTokens = 64;    // tokens of one dz block
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
  size_t err, dz, bias, dw, total;  // byte offsets
};

cudaError_t launch_route_products_tc(const RouteBackwardArgs& a, const RouteBackwardPlan& p,
                                     cudaStream_t s);
constexpr int kRbTcCols = 128;   // columns and tokens of one tile
constexpr int kRbTcTokens = 128;

}  // namespace moe
