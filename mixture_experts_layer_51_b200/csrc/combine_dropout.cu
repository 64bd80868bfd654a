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
// One token's row is owned by the lanes of one CTA, so the k gate gradients
// are a fixed-order sum and nothing is atomic; every permuted row belongs to
// one (token, slot), so the scatter of d_o writes each row once.
//
// Bound by HBM: the kept rows of o, y or dy, the residual, d_o, each once.
// Measured on one B200 in a graph (floors at 6.56 TB/s in brackets), p = 0.1,
// bf16: forward with residual 8192 x 4096 top-2 42.4 us (40.9), top-4 61.5
// (61.4), 16384 x 2048 top-8 100.7 us (102.4); backward 8192 x 4096 top-2 54.6 us
// (51.1; 53.5 without dropout, so the generator hides behind the copies), top-4
// 97.4 (92.1), 16384 x 2048 top-8 180 us (174).  fp32, 8192 x 4096: forward with
// residual top-2 78.9 us (81.8), top-4 117 (123), top-8 195 (205); backward top-2
// 103 (102), top-4 187 (184), top-8 370 (348).
// The backward pass writes the rows of d_o that a kept slot owns, and its time
// is that of these rows: a reader that takes whole 128-row blocks has to clear
// the others itself (at most 127 rows an expert).
// What made the difference: all loads of a sweep before any
// arithmetic (156 -> 106 us on the top-8 forward), plain instead of
// evict-first loads (192 -> 185 us on the top-8 backward), and four sweeps a
// warp (57.5 -> 55.8 us on 8192 x 4096).  More resident warps through fewer
// registers were slower (60 -> 70 us).

#include "moe_internal.cuh"
#include "philox.cuh"

namespace moe {
namespace {

constexpr int kCdWarps = 8;

// Eight consecutive elements: their bytes, as loaded and stored, and in fp32.
// load() takes the read-only path, for what nobody writes during the kernel;
// load_plain() is for the residual, which y may be.
template <bool BF16>
struct Chunk;
template <>
struct Chunk<true> {
  static constexpr int kBytes = 16;
  uint4 v;
  __device__ __forceinline__ void load(const char* p) {
    v = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void load_plain(const char* p) {
    v = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  // Elements 2 i and 2 i + 1 stay where the low and high half of m[i] are all
  // ones, and become zero where they are zeros.
  __device__ __forceinline__ void mask(const uint32_t (&m)[4]) {
    v.x &= m[0], v.y &= m[1], v.z &= m[2], v.w &= m[3];
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(char* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Chunk<false> {
  static constexpr int kBytes = 32;
  float4 a, b;
  __device__ __forceinline__ void load(const char* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_plain(const char* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void mask(const uint32_t (&m)[4]) {
    a.x = m[0] & 1u ? a.x : 0.f;
    a.y = m[0] >> 31 ? a.y : 0.f;
    a.z = m[1] & 1u ? a.z : 0.f;
    a.w = m[1] >> 31 ? a.w : 0.f;
    b.x = m[2] & 1u ? b.x : 0.f;
    b.y = m[2] >> 31 ? b.y : 0.f;
    b.z = m[3] & 1u ? b.z : 0.f;
    b.w = m[3] >> 31 ? b.w : 0.f;
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  static __device__ __forceinline__ void store(char* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// m[i]: all ones in the low and high half where elements 2 i and 2 i + 1 of
// the words' group are kept, zeros where they are dropped.
__device__ __forceinline__ void keep_masks(const uint32_t (&w)[4], uint32_t threshold,
                                           uint32_t (&m)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // threshold - 1 - half is negative where half >= threshold; its sign
    // fills both bytes of the half.
    const int lo = static_cast<int>(threshold - 1) - static_cast<int>(w[i] & 0xffffu);
    const int hi = static_cast<int>(threshold - 1) - static_cast<int>(w[i] >> 16);
    asm("prmt.b32 %0, %1, %2, 0xffbb;" : "=r"(m[i]) : "r"(lo), "r"(hi));
  }
}

// A token's row belongs to L lanes of a warp (8 or 32), or of each of
// 1 << warp_bits warps of a CTA (L = 32 only): this thread's token, which of
// the token's warps it is in, and its lane there.
struct Place {
  int64_t t;
  int part, lane;
};
__host__ __device__ constexpr int tokens_per_cta(int L, int warp_bits) {
  return kCdWarps * 32 / L >> warp_bits;
}
template <int L>
__device__ __forceinline__ Place place(int warp_bits) {
  const int thread = threadIdx.x, group = thread / L;
  return {static_cast<int64_t>(blockIdx.x) * tokens_per_cta(L, warp_bits) + (group >> warp_bits),
          group & ((1 << warp_bits) - 1), thread % L};
}

// The token's rows and gates, in every lane of it (row -1: no such slot, as
// for tokens past the last).  Whole warps call this.
template <int KJ, int L>
__device__ __forceinline__ void slots(const int32_t* pos, const float* gate, const Place& at,
                                      int T, int k, int (&row)[KJ], float (&g)[KJ]) {
  const bool in = at.t < T && at.lane < k;
  const int pl = in ? pos[at.t * k + at.lane] : -1;
  const float gl = in ? gate[at.t * k + at.lane] : 0.f;
#pragma unroll
  for (int j = 0; j < KJ; ++j) {
    row[j] = __shfl_sync(0xffffffffu, pl, j, L);
    g[j] = __shfl_sync(0xffffffffu, gl, j, L);
  }
}

// KJ = slots this instantiation handles (2, 4 or 8, the least that k fits); CH =
// 8-element chunks of each row per lane and iteration: every load of an
// iteration is issued before any arithmetic (the generator's, too, runs while
// they are on their way).
template <bool BF16, int KJ, int CH, int L>
__global__ void __launch_bounds__(kCdWarps * 32)
    combine_dropout_kernel(const void* __restrict__ o, const int32_t* __restrict__ pos,
                           const float* __restrict__ gate, const void* residual,
                           const uint64_t* __restrict__ rng, uint32_t threshold, float scale,
                           int T, int d, int k, int warp_bits, void* y) {
  pdl_wait();
  pdl_trigger();
  constexpr uint32_t B = Chunk<BF16>::kBytes;
  const Place at = place<L>(warp_bits);
  const int64_t t = at.t;
  const uint32_t n8 = d / 8;
  uint64_t seed = 0, offset = 0;
  if (threshold) seed = rng[0], offset = rng[1];
  int row[KJ];
  float g[KJ];
  const char* from[KJ];
  slots<KJ, L>(pos, gate, at, T, k, row, g);
  if (t >= T) return;
#pragma unroll
  for (int j = 0; j < KJ; ++j) {
    g[j] *= scale;
    from[j] = static_cast<const char*>(o) + static_cast<int64_t>(row[j]) * n8 * B;
  }
  const char* rest = static_cast<const char*>(residual) + t * n8 * B;
  char* to = static_cast<char*>(y) + t * n8 * B;
  const PhiloxKeys keys = philox_keys(seed);
  for (uint32_t c0 = at.part * L * CH + at.lane; c0 < n8; c0 += L * CH << warp_bits) {
    const uint64_t at_c = static_cast<uint64_t>(c0) * B;
    Chunk<BF16> v[KJ][CH], res[CH];
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      const bool in = c0 + h * L < n8;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        if (row[j] >= 0 && in)
          v[j][h].load(from[j] + at_c + h * L * B);
        else
          v[j][h].zero();
      }
      if (residual && in)
        res[h].load_plain(rest + at_c + h * L * B);
      else
        res[h].zero();
    }
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      if (c0 + h * L >= n8) break;
      float acc[8] = {}, f[8];
      uint32_t w[4];
      if (threshold) philox4x32_10(t * n8 + c0 + h * L, offset, keys, w);
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        if (row[j] < 0) continue;  // absent slots add nothing
        v[j][h].unpack(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(g[j], f[i], acc[i]);
      }
      if (threshold) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = dropout_kept(w, i, threshold) ? acc[i] : 0.f;
      }
      if (residual) {
        res[h].unpack(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
      }
      Chunk<BF16>::store(to + at_c + h * L * B, acc);
    }
  }
}

// Adds `v` over each group of L lanes (at least N): afterwards lane l of a
// group holds the total of v[l / (L / N)], each added in an order that is
// always the same.
template <int N, int L>
__device__ __forceinline__ float reduce_lanes(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int s = L / 2;
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

template <bool BF16, int KJ, int CH, int L>
__global__ void __launch_bounds__(kCdWarps * 32)
    combine_dropout_backward_kernel(const void* __restrict__ dy, const void* __restrict__ o,
                                    const int32_t* __restrict__ pos,
                                    const float* __restrict__ gate,
                                    const uint64_t* __restrict__ rng, uint32_t threshold,
                                    float scale, int T, int d, int k, int warp_bits,
                                    void* __restrict__ d_o, float* __restrict__ dgate) {
  __shared__ float part[kCdWarps][KJ];
  pdl_wait();
  pdl_trigger();
  const Place at = place<L>(warp_bits);
  constexpr uint32_t B = Chunk<BF16>::kBytes;
  const int warp = threadIdx.x >> 5, lane = at.lane;
  const int64_t t = at.t;
  const uint32_t n8 = d / 8;
  float dot[KJ] = {}, g[KJ];
  int row[KJ];
  uint64_t seed = 0, offset = 0;
  if (threshold) seed = rng[0], offset = rng[1];
  slots<KJ, L>(pos, gate, at, T, k, row, g);
  if (t < T) {
    const char* from[KJ];
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      g[j] *= scale;
      from[j] = static_cast<const char*>(o) + static_cast<int64_t>(row[j]) * n8 * B;
    }
    const char* up_row = static_cast<const char*>(dy) + t * n8 * B;
    char* to = static_cast<char*>(d_o);
    const PhiloxKeys keys = philox_keys(seed);
    for (uint32_t c0 = at.part * L * CH + at.lane; c0 < n8; c0 += L * CH << warp_bits) {
      const uint64_t at_c = static_cast<uint64_t>(c0) * B;
      Chunk<BF16> v[KJ][CH], up[CH];
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (c0 + h * L >= n8) break;
        up[h].load(up_row + at_c + h * L * B);
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          if (row[j] >= 0) v[j][h].load(from[j] + at_c + h * L * B);
      }
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (c0 + h * L >= n8) break;
        // Dropped elements become zero in dy and in o (what o holds there is
        // left out: 0 times it need not be 0).
        uint32_t m[4];
        if (threshold) {
          uint32_t w[4];
          philox4x32_10(t * n8 + c0 + h * L, offset, keys, w);
          keep_masks(w, threshold, m);
          up[h].mask(m);
        }
        float a[8];
        up[h].unpack(a);
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          if (row[j] < 0) continue;
          if (threshold) v[j][h].mask(m);
          float f[8];
          v[j][h].unpack(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(a[i], f[i], dot[j]);
            f[i] = g[j] * a[i];  // g carries the scale
          }
          Chunk<BF16>::store(to + (from[j] - static_cast<const char*>(o)) + at_c + h * L * B, f);
        }
      }
    }
  }
  // The row's dot products: over the lanes, then over the warps that share it.
  const float sum = scale * reduce_lanes<KJ, L>(dot);
  constexpr int W = L / KJ;  // lanes that hold the same total
  if (warp_bits == 0) {
    if (t < T && lane % W == 0 && lane / W < k)
      dgate[t * k + lane / W] = pos[t * k + lane / W] >= 0 ? sum : 0.f;
    return;
  }
  if (lane % W == 0) part[warp][lane / W] = sum;
  __syncthreads();
  if (t < T && at.part == 0 && lane < k) {
    float total = 0.f;
    for (int i = 0; i < 1 << warp_bits; ++i) total += part[warp + i][lane];
    dgate[t * k + lane] = pos[t * k + lane] >= 0 ? total : 0.f;
  }
}

// log2 of the warps a row, for kernels whose warps sweep 32 `ch` chunks of a
// row at a time: as many as leave each four sweeps; and where the tokens are
// too few to fill the GPU (eight warps on each of 148 SMs), as many as leave
// each one.
int pick_warp_bits(int T, int d, int ch) {
  const int sweeps = (d / 8 + 32 * ch - 1) / (32 * ch);
  int bits = 0;
  while ((1 << bits) < kCdWarps &&
         (sweeps >= 8 << bits ||
          (static_cast<int64_t>(T) << bits < 148 * kCdWarps && sweeps >= 2 << bits)))
    ++bits;
  return bits;
}

// Rows of at most 16 chunks take eight lanes of a warp, so that its other
// lanes work on other rows (100000 x 64, top-2, bf16: forward 39.7 -> 10.1 us
// without a residual, 10.6 with one, backward 48.0 -> 12.6; with a row width known only at run time the wide rows
// lose: 98 -> 115 us on 16384 x 2048 top-8).
bool narrow(int d) { return d <= 128; }

template <bool BACKWARD, bool BF16, int KJ, int CH, int L>
cudaError_t launch(const CombineDropoutArgs& a, cudaStream_t s) {
  const int warp_bits = L == 32 ? pick_warp_bits(a.T, a.d, CH) : 0;
  const int tokens = tokens_per_cta(L, warp_bits);
  const dim3 grid((static_cast<unsigned>(a.T) + tokens - 1) / tokens), block(kCdWarps * 32);
  if constexpr (BACKWARD)
    return launch_kernel(combine_dropout_backward_kernel<BF16, KJ, CH, L>, grid, block, 0, s, 1,
                         true, a.dy, a.o, a.pos, a.gate, a.rng, a.threshold, a.scale, a.T, a.d,
                         a.k, warp_bits, a.d_o, a.dgate);
  else
    return launch_kernel(combine_dropout_kernel<BF16, KJ, CH, L>, grid, block, 0, s, 1, true, a.o,
                         a.pos, a.gate, a.residual, a.rng, a.threshold, a.scale, a.T, a.d, a.k,
                         warp_bits, a.y);
}

// Two chunks a lane and sweep where the registers hold them: of up to two
// slots in bf16, in the backward pass of up to four (8192 x 4096 top-4: 111 us
// with one chunk, 96 with two; forward 60.4 and 62.2).  A kernel for four
// slots of its own, since the absent ones of eight hold registers and issue
// slots (8192 x 4096 top-4: 66 and 115 us; 16384 x 512 top-4 forward 21.2 us
// against 15.6).
template <bool BACKWARD, bool BF16>
cudaError_t pick(const CombineDropoutArgs& a, cudaStream_t s) {
  constexpr int C2 = BF16 ? 2 : 1, C4 = BF16 && BACKWARD ? 2 : 1;
  if (narrow(a.d))
    return a.k <= 2   ? launch<BACKWARD, BF16, 2, 1, 8>(a, s)
           : a.k <= 4 ? launch<BACKWARD, BF16, 4, 1, 8>(a, s)
                      : launch<BACKWARD, BF16, kMaxK, 1, 8>(a, s);
  return a.k <= 2   ? launch<BACKWARD, BF16, 2, C2, 32>(a, s)
         : a.k <= 4 ? launch<BACKWARD, BF16, 4, C4, 32>(a, s)
                    : launch<BACKWARD, BF16, kMaxK, 1, 32>(a, s);
}

}  // namespace

cudaError_t launch_combine_dropout(const CombineDropoutArgs& a, moe_dtype dtype, cudaStream_t s) {
  return dtype == MOE_BF16 ? pick<false, true>(a, s) : pick<false, false>(a, s);
}

cudaError_t launch_combine_dropout_backward(const CombineDropoutArgs& a, moe_dtype dtype,
                                            cudaStream_t s) {
  return dtype == MOE_BF16 ? pick<true, true>(a, s) : pick<true, false>(a, s);
}

}  // namespace moe
