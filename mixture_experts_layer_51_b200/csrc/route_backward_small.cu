// The router's backward pass for small batches, in one launch.
//
// At these sizes the pass is bound by the host's launches and by round trips
// to memory, not by bytes or products.  So every CTA (32 columns) makes dz of
// all tokens again for itself, in shared memory, and both products follow on
// fp32 FMA with nothing shared between CTAs: no workspace, no ranges to add.
// x, W_g and dx_acc are asked for before dz is made.
//
// Register tiles as in route_backward.cu: 4 columns x 4 experts over the
// tokens for dW_g (the tokens shared out over eight groups of threads, added
// up in order), 2 tokens x 4 columns over the experts for dx.
//
// Where it is taken: up to 256 tokens and 4096 dz values (experts rounded up
// to 8, 16, 32 or 64), and no more CTAs than SMs.  Measured in a graph on one
// B200 against the two launches of route_backward.cu (bf16): 256 x 64, 4
// experts 5.7 us (7.1); 256 x 4096, 8 experts 6.4 (8.9), 16 experts 8.2 (9.1);
// 128 x 4096, 32 experts 7.9 (10.0); 64 x 4096, 64 experts 9.5 (10.3); past the
// rule 256 x 1024, 32 experts 11.0 (10.4), 128 x 1024, 64 experts 11.8 (10.5),
// where the products' shared memory reads bound it, and 256 x 8192, 8 experts
// 11.3 (9.0), with two CTAs an SM.  The host saves 2.5 us a call.

#include "route_backward.cuh"

namespace moe {
namespace {

constexpr int kTokens = kRbSmallTokens;
constexpr int kParts = 4;                   // threads of a token while dz is made
constexpr int kThreads = kTokens * kParts;
constexpr int kCols = 32;
constexpr int kGroups = 8;                  // of threads that share out dW_g's tokens

template <int EP>
struct Smem {
  // dz; later the token groups' parts of dW_g, [kGroups][kCols][EP].
  float z[kTokens][EP + 4];
  union {
    float x[kTokens][kCols];
    struct {
      float part[2][kParts][kTokens];
      int32_t sel[kMaxK][kTokens];
      float term[kMaxK][kTokens];
    };
  };
  float w[EP][kCols + 4];
  __align__(16) float f[kMaxE];
};
static_assert(kTokens * 4 >= kGroups * kCols, "the parts of dW_g fit in dz's place");

// Q consecutive floats of shared memory in 16-byte (Q = 2: 8-byte) pieces:
// rows of dz start 16 bytes apart round the banks, so a warp's do not collide.
template <int Q>
__device__ __forceinline__ void get(const float* from, float (&v)[Q]) {
  constexpr int N = Q < 4 ? Q : 4;
#pragma unroll
  for (int i = 0; i < Q; i += N) {
    if (N == 4) {
      const float4 x = *reinterpret_cast<const float4*>(from + i);
      v[i] = x.x, v[i + 1] = x.y, v[(i + 2) % Q] = x.z, v[(i + 3) % Q] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(from + i);
      v[i] = x.x, v[i + 1] = x.y;
    }
  }
}
template <int Q>
__device__ __forceinline__ void put(float* to, const float (&v)[Q]) {
  constexpr int N = Q < 4 ? Q : 4;
#pragma unroll
  for (int i = 0; i < Q; i += N) {
    if (N == 4)
      *reinterpret_cast<float4*>(to + i) =
          make_float4(v[i], v[i + 1], v[(i + 2) % Q], v[(i + 3) % Q]);
    else
      *reinterpret_cast<float2*>(to + i) = make_float2(v[i], v[i + 1]);
  }
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if (BF16) {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
template <bool BF16>
__device__ __forceinline__ float4 load4(const void* p, int64_t at) {
  if (BF16) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
  }
  return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t at, float4 v) {
  if (BF16)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + at) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = v;
}

template <bool BF16, int EP>
__global__ void __launch_bounds__(kThreads, 1)
    route_small_kernel(const RouteBackwardArgs a, int32_t* __restrict__ err) {
  constexpr int Q = EP / kParts, EG = EP / 4;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<EP>& sm = *reinterpret_cast<Smem<EP>*>(smem_raw);
  const int tid = threadIdx.x, c0 = blockIdx.x * kCols, cols = min(kCols, a.d - c0);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && tid == 0) *err = 0;

  // ------------------------------------------------------- what is needed
  // x: a row's eight columns a thread (columns come in eights).
  const int xr = tid / 4, xc = tid % 4 * 8;
  float xv[8] = {};
  if (a.dWg && xr < a.T && xc < cols && (!a.mask || a.mask[xr]))
    load8<BF16>(a.x, static_cast<int64_t>(xr) * a.d + c0 + xc, xv);
  // dx_acc: two rows' four columns a thread.
  const int cg = tid % 8, row = tid / 8 * 2;
  const bool in = 4 * cg < cols;
  float4 out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    out[i] = a.dx && a.dx_acc && in && row + i < a.T
                 ? load4<BF16>(a.dx_acc, static_cast<int64_t>(row + i) * a.d + c0 + 4 * cg)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.dx)
    for (int i = tid; i < kCols * EP; i += kThreads) {
      const int c = i / EP, e = i % EP;
      float v = 0.f;
      if (c < cols && e < a.E) {
        const int64_t at = static_cast<int64_t>(c0 + c) * a.E + e;
        v = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.Wg)[at])
                 : static_cast<const float*>(a.Wg)[at];
      }
      sm.w[e][c] = v;
    }

  // ------------------------------------------------------------------- dz
  {
    const int tok = tid % kTokens, q = tid / kTokens, e0 = q * Q;
    const bool here = tok < a.T;
    const bool all = a.dgate && a.gating == MOE_GATE_SOFTMAX_TOPK;
    const int n = a.counts ? *a.tokens : 0;
    const float dloss = a.counts && a.dloss ? *a.dloss : 1.f;
    const int count = a.counts && tid < a.E ? a.counts[tid] : 0;
    const bool live = here && (!a.mask || a.mask[tok]);
    float p[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i)
      p[i] = here && (a.counts || all) && e0 + i < a.E
                 ? a.scores[static_cast<int64_t>(e0 + i) * a.T + tok]
                 : 0.f;
    int sel[2];
    float g[2], dg[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int j = q + kParts * s;
      const bool use = here && a.dgate && j < a.k;
      const int64_t at = static_cast<int64_t>(tok) * a.k + j;
      sel[s] = use ? a.idx[at] : -1;
      g[s] = use ? a.gate[at] : 0.f;
      dg[s] = use ? a.dgate[at] : 0.f;
    }
    const bool loss = n > 0;
    if (tid < kMaxE)
      sm.f[tid] = loss ? static_cast<float>(count) / (static_cast<float>(n) * a.k) : 0.f;
    const float c = loss ? a.coef * dloss * a.E / n : 0.f;
    float z[Q] = {};
    put(&sm.z[tok][e0], z);
#pragma unroll
    for (int i = 0; i < Q; ++i)
      if (!live) p[i] = 0.f;  // whatever a padding token holds
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (!live) g[s] = dg[s] = 0.f;
    __syncthreads();
    float mean = 0.f, f[Q];
    get(&sm.f[e0], f);
#pragma unroll
    for (int i = 0; i < Q; ++i) mean = fmaf(f[i], p[i], mean);
    sm.part[0][q][tok] = fmaf(g[0], dg[0], g[1] * dg[1]);
    sm.part[1][q][tok] = mean;
    __syncthreads();
    float total = 0.f;
    mean = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      total += sm.part[0][i][tok], mean += sm.part[1][i][tok];
    if (a.dgate) {
      // The first of the slots that name an expert adds them all, in order.
      const float rest = a.gate_scale == 1.f ? total : total / a.gate_scale;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        sm.sel[q + kParts * s][tok] = live && sel[s] < a.E ? sel[s] : -1;
        sm.term[q + kParts * s][tok] = all ? g[s] * dg[s] : g[s] * (dg[s] - rest);
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int mine = sm.sel[q + kParts * s][tok];
        if (mine < 0) continue;
        float sum = 0.f;
        bool first = true;
#pragma unroll
        for (int j = 0; j < kMaxK; ++j) {
          const bool same = sm.sel[j][tok] == mine;
          if (same && j < q + kParts * s) first = false;
          if (same) sum += sm.term[j][tok];
        }
        if (first) sm.z[tok][mine] = sum;
      }
    }
    __syncthreads();
    if (live && (loss || all)) {
      get(&sm.z[tok][e0], z);
      get(&sm.f[e0], f);
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        if (loss) z[i] = fmaf(c * p[i], f[i] - mean, z[i]);
        if (all) z[i] = fmaf(-p[i], total, z[i]);
        if (e0 + i >= a.E) z[i] = 0.f;
      }
      put(&sm.z[tok][e0], z);
    }
    __syncthreads();
  }
  if (a.dWg) {
    float4* to = reinterpret_cast<float4*>(&sm.x[xr][xc]);
    to[0] = make_float4(xv[0], xv[1], xv[2], xv[3]);
    to[1] = make_float4(xv[4], xv[5], xv[6], xv[7]);
    __syncthreads();
  }

  // ------------------------------------------------------------- products
  if (a.dx && in && row < a.T) {
#pragma unroll 4
    for (int e = 0; e < EP; e += 4) {
      float zs[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(&sm.z[row + i][e]);
        zs[i][0] = v.x, zs[i][1] = v.y, zs[i][2] = v.z, zs[i][3] = v.w;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 w = *reinterpret_cast<const float4*>(&sm.w[e + u][4 * cg]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          out[i].x = fmaf(zs[i][u], w.x, out[i].x);
          out[i].y = fmaf(zs[i][u], w.y, out[i].y);
          out[i].z = fmaf(zs[i][u], w.z, out[i].z);
          out[i].w = fmaf(zs[i][u], w.w, out[i].w);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (row + i < a.T)
        store4<BF16>(a.dx, static_cast<int64_t>(row + i) * a.d + c0 + 4 * cg, out[i]);
  }
  if (a.dbias && blockIdx.x == 0)  // one warp an expert
    for (int e = tid / 32; e < a.E; e += kThreads / 32) {
      float s = 0.f;
      for (int t = tid % 32; t < a.T; t += 32) s += sm.z[t][e];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (tid % 32 == 0) a.dbias[e] = s;
    }
  if (!a.dWg) return;
  // Neighbouring threads take neighbouring experts, so that the parts below
  // are stored without bank conflicts.
  const int eg = tid % EG, wg = tid / EG % 8, tg = tid / (8 * EG);
  float acc[4][4] = {};
  if (tg < kGroups)
#pragma unroll 4
    for (int t = tg; t < a.T; t += kGroups) {
      const float4 x4 = *reinterpret_cast<const float4*>(&sm.x[t][4 * wg]);
      const float4 z4 = *reinterpret_cast<const float4*>(&sm.z[t][4 * eg]);
      const float xs[4] = {x4.x, x4.y, x4.z, x4.w}, zs[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(xs[i], zs[e], acc[i][e]);
    }
  __syncthreads();  // dz has been read
  float* part = &sm.z[0][0];
  if (tg < kGroups)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(part + (tg * kCols + 4 * wg + i) * EP + 4 * eg) =
          make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  __syncthreads();
  for (int i = tid; i < cols * a.E; i += kThreads) {
    const int c = i / a.E, e = i % a.E;
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) s += part[(g * kCols + c) * EP + e];
    a.dWg[static_cast<int64_t>(c0) * a.E + i] = s;
  }
}

template <bool BF16, int EP>
cudaError_t launch(const RouteBackwardArgs& a, int32_t* err, cudaStream_t s) {
  const auto kern = route_small_kernel<BF16, EP>;
  constexpr int smem = sizeof(Smem<EP>);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const int ctas = a.dx || a.dWg ? (a.d + kCols - 1) / kCols : 1;
  return launch_kernel(kern, dim3(ctas), dim3(kThreads), smem, s, 1, true, a, err);
}

}  // namespace

bool route_backward_is_small(int T, int d, int E) {
  const int EP = E <= 8 ? 8 : E <= 16 ? 16 : E <= 32 ? 32 : 64;
  return T <= kTokens && T * EP <= 4096 && (d + kCols - 1) / kCols <= kRbSms;
}

cudaError_t launch_route_backward_small(const RouteBackwardArgs& a, moe_dtype dtype, int32_t* err,
                                        cudaStream_t s) {
  if (dtype == MOE_BF16)
    return a.E <= 8    ? launch<true, 8>(a, err, s)
           : a.E <= 16 ? launch<true, 16>(a, err, s)
           : a.E <= 32 ? launch<true, 32>(a, err, s)
                       : launch<true, 64>(a, err, s);
  return a.E <= 8    ? launch<false, 8>(a, err, s)
         : a.E <= 16 ? launch<false, 16>(a, err, s)
         : a.E <= 32 ? launch<false, 32>(a, err, s)
                     : launch<false, 64>(a, err, s);
}

}  // namespace moe
