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
// Small batches go to route_backward_small.cu in one launch; the others take
// two launches or three.  (1) dz for every token, and its column sums per
// block of tokens.  (2) Both products in one pass over x: a CTA owns a block
// of columns and a range of tokens, so each x element is read once, each dx
// element written once, and dW_g of the block stays on the chip until the
// range is done (bf16: tensor cores, route_backward_tc.cu; fp32: FMA, here).
// (3) With many ranges, their sum; with few, the last range of a column block
// to finish adds all of the block's.  Either goes in order, and one warp an
// expert adds the dz blocks' column sums: no sum depends on scheduling (no
// floating-point atomics).
//
// dz is a launch of its own because every column block needs it: 5.6 MB of
// scores and gates in, 128 to 384 bytes a token out (bf16 terms), 7 to 8 us for
// 16384 tokens of 64 experts beside the products' first loads, of which about
// 3 are its arithmetic.  Blocks of 32 tokens with eight threads a token beat
// 64 with four (48.3 -> 46.7 us for the whole pass), and 64 registers a thread
// beat 32 (46.7 -> 44.7 us).

#include "route_backward.cuh"

namespace moe {
namespace {

constexpr int kDzParts = 8;        // threads of a token in the dz kernel
constexpr int kDzThreads = kDzParts * kRbTokens;
constexpr int kCols = 64;          // fp32 products: columns of one CTA,
constexpr int kTile = 64;          // tokens of one tile
constexpr int kThreads = 256;

// Token ranges for `cols` column blocks: the number that needs the fewest
// tile times, where a wave of kRbSms CTAs takes the tiles of its longest
// range and about five more for its start and its end.
int pick_ranges(int cols, int tiles, int per_sm) {
  int best = 1;
  int64_t best_cost = INT64_MAX;
  const int slots = kRbSms * per_sm;
  const int most = tiles < 2 * slots / cols + 1 ? tiles : 2 * slots / cols + 1;
  for (int r = 1; r <= most; ++r) {
    const int64_t waves = (static_cast<int64_t>(cols) * r + slots - 1) / slots;
    const int64_t cost = waves * ((tiles + r - 1) / r + 5);
    if (cost < best_cost) best_cost = cost, best = r;
  }
  return best;
}

// The ranges of dW_g are added by the last CTA of a column block, or by a
// launch over all SMs.  The launch is quicker on the GPU from about five
// ranges on (in a graph, with and without it: 16384 x 2048, 64 experts, 9
// ranges, bf16 40.2 and 42.7 us; 1001 x 1032, 8 experts, 8 ranges, bf16 8.3 and
// 9.8; 2048 x 1024, 8 experts, 16 ranges, fp32 9.5 and 11.6; 16384 x 64, 64
// experts, 128 ranges, bf16 14.2 and 52; at four ranges both take as long), but
// costs the host 2 us, and a call from Python takes the host about 16 us
// without it.  So a pass that the GPU is through with in that time does without
// (1001 x 1032 above: 18.3 us a call with the launch, 16.2 without; 2048 x 1024:
// 18.3 and 16.3), as long as one CTA has no more than 20 ranges to add.  How
// long the GPU takes goes by x's bytes and, with many experts, by the products
// (us a call with the launch and without):
//   bytes: fp32, 8 experts, 2048 x 2048 (16 MB) 18.1 and 16.2, 4096 x 1536 (24
//   MB) 18.5 and 20.1; bf16, 16 experts, 6000 x 1024 (12 MB) 18.8 and 18.1, 8192
//   x 1024 (16 MB) 18.6 and 19.7: even at about 14 MB, where a graph gains 2 to
//   5 us already;
//   products, fp32: 2048 x 1024, 16 experts (33 M) 18.2 and 16.4, 4096 x 768, 16
//   experts (50 M) 18.4 and 21.8, 1001 x 1032, 64 experts (66 M) 18.3 and 22.3;
//   bf16, which are quicker, with the ranges' sum the longer part: 1001 x 1032, 64
//   experts (66 M) 18.4 and 16.4, 2048 x 1024, 64 experts (134 M) 18.6 and 18.4,
//   4096 x 768, 64 experts (201 M) 18.7 and 20.1.
constexpr int kFewRanges = 4;
constexpr int kPassingRanges = 20;
constexpr int64_t kSummingBytes = 14 << 20;                          // of x
constexpr int64_t kSummingFp32 = 42000000, kSummingBf16 = 112000000;  // T d E

bool sum_by_launch(int ranges, int T, int d, int E, bool tc) {
  const int64_t elements = static_cast<int64_t>(T) * d;
  return ranges > kPassingRanges ||
         (ranges > kFewRanges && (elements * (tc ? 2 : 4) >= kSummingBytes ||
                                  elements * E >= (tc ? kSummingBf16 : kSummingFp32)));
}

RouteBackwardPlan make_plan(int T, int d, int E, moe_dtype dtype) {
  RouteBackwardPlan p{};
  const bool tc = dtype == MOE_BF16;
  p.EP = E <= 8 ? 8 : E <= 16 ? 16 : E <= 32 ? 32 : 64;
  p.blocks = (T + kRbTokens - 1) / kRbTokens;
  const int cols = tc ? kRbTcCols : kCols, tile = tc ? kRbTcTokens : kTile;
  p.cols = (d + cols - 1) / cols;
  p.tiles = (T + tile - 1) / tile;
  p.ranges = T > 0 ? pick_ranges(p.cols, p.tiles, tc ? 1 : 2) : 0;
  p.many = sum_by_launch(p.ranges, T, d, E, tc);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  p.err = take(sizeof(int32_t));
  p.tickets = take(sizeof(uint32_t) * p.cols);
  const size_t row = tc ? 128 * dz_terms(E).blocks : sizeof(float) * p.EP;
  p.dz = take(row * T);
  p.bias = take(sizeof(float) * kMaxE * p.blocks);
  p.dw = take(tc && dz_terms(E).blocks == 3 && !p.many
                  ? static_cast<size_t>(kRbPartBytes) * p.cols * p.ranges
                  : sizeof(float) * d * E * p.ranges);
  p.total = at;
  return p;
}

// v = hi + mid + lo, each with a bf16's eight significant bits (in the upper
// half of its fp32 pattern).  Each term is cut from just below what is left, so
// that the next has something to hold: every term of a value other than zero
// has that value's sign and is not zero, and an infinity in x or W_g times the
// three adds up to what it gives with v (with terms of zero or of both signs,
// NaN).  Infinities and NaN are all three terms.  Exact down to 2^-100; further
// down a term may be too small for bf16 and is its least value then, 2^-133.
struct Terms {
  uint32_t hi, mid, lo;
};
__device__ __forceinline__ Terms split(float v) {
  const uint32_t u = __float_as_uint(v), size = u & 0x7fffffffu;
  if (size == 0 || size >= 0x7f800000u) {
    const uint32_t same = size > 0x7f800000u ? u | 0x00400000u : u;  // NaN in the upper half
    return {same, same, same};
  }
  const uint32_t least = (u & 0x80000000u) | 0x00010000u;
  Terms t;
  t.hi = (u - 1) & 0xffff0000u;
  const float rest = v - __uint_as_float(t.hi);
  t.mid = (__float_as_uint(rest) - 1) & 0xffff0000u;
  t.lo = __float_as_uint(rest - __uint_as_float(t.mid));
  if (size < 0x18000000u) {  // 2^-79: far above where a term runs out
    if (!(t.hi & 0x7fff0000u)) t.hi = least;
    if (!(t.mid & 0x7fff0000u)) t.mid = least;
    if (!(t.lo & 0x7fff0000u)) t.lo = least;
  }
  return t;
}
// The upper halves of two words, `a`'s below `b`'s.
__device__ __forceinline__ uint32_t upper_halves(uint32_t a, uint32_t b) {
  return __byte_perm(a, b, 0x7632);
}

// dz of 32 tokens, eight threads a token (each an eighth of the experts, kept
// in registers so that the scores are read once), and its column sums.  TC:
// dz leaves as bf16 terms, else as fp32 rows of EP; either way by way of
// shared memory, in whole 16-byte pieces of contiguous rows.  Q: experts a
// thread has room for (an eighth of E, rounded up to a power of two).
template <bool TC, int Q>
__global__ void __launch_bounds__(kDzThreads, 4)
    route_dz_kernel(const RouteBackwardArgs a, int EP, DzTerms terms, void* __restrict__ dz,
                    float* __restrict__ bias_part, int32_t* __restrict__ err,
                    uint32_t* __restrict__ tickets, int ntickets) {
  // Rows start 16 bytes further round the banks than the one before.
  constexpr int LD = 64 * 3 + 8;
  __shared__ float z[kRbTokens][kMaxE + 1];
  __shared__ __align__(16) __nv_bfloat16 rows_s[TC ? kRbTokens * LD : 8];
  __shared__ float f[kMaxE];
  __shared__ float part[2][kDzParts][kRbTokens];
  __shared__ int32_t sel_s[kMaxK][kRbTokens];
  __shared__ float term_s[kMaxK][kRbTokens];
  __shared__ float sum_s[4][kMaxE];
  const int tid = threadIdx.x, tok = tid % kRbTokens, q = tid / kRbTokens;
  const int t0 = blockIdx.x * kRbTokens, t = t0 + tok;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) {
    if (tid == 0) *err = 0;
    for (int i = tid; i < ntickets; i += kDzThreads) tickets[i] = 0;
  }
  // Every load before the first use of any (a padding token's values are
  // loaded and dropped, which is quicker than to wait for its mask).
  const bool in = t < a.T;
  const bool all = a.dgate && a.gating == MOE_GATE_SOFTMAX_TOPK;
  const int n = a.counts ? *a.tokens : 0;
  const float dloss = a.counts && a.dloss ? *a.dloss : 1.f;
  const int count = a.counts && tid < a.E ? a.counts[tid] : 0;
  const bool live = in && (!a.mask || a.mask[t]);
  const int per = (a.E + kDzParts - 1) / kDzParts, e0 = q * per;  // this thread's experts: e0 .. e0 + per - 1
  const int mine = min(per, a.E - e0);
  float p[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i)
    p[i] = in && (a.counts || all) && i < mine
               ? a.scores[static_cast<int64_t>(e0 + i) * a.T + t]
               : 0.f;
  // The token's slot q.
  static_assert(kMaxK <= kDzParts, "a slot a thread");
  const bool slot = in && a.dgate && q < a.k;
  const int64_t at = static_cast<int64_t>(t) * a.k + q;
  const int sel = slot ? a.idx[at] : -1;
  float g = slot ? a.gate[at] : 0.f, dg = slot ? a.dgate[at] : 0.f;
  const bool loss = n > 0;
  if (tid < kMaxE)
    f[tid] = loss ? static_cast<float>(count) / (static_cast<float>(n) * a.k) : 0.f;
  const float c = loss ? a.coef * dloss * a.E / n : 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i)
    if (i < mine) z[tok][e0 + i] = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i)
    if (!live) p[i] = 0.f;
  if (!live) g = dg = 0.f;
  // What no expert's term fills stays zero (with three blocks of terms every
  // place of a row that is read is written below, or here).
  if (TC && a.E < 64)
    for (int i = tid; i < kRbTokens * LD / 8; i += kDzThreads)
      reinterpret_cast<uint4*>(rows_s)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  float mean = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i)
    if (i < mine) mean = fmaf(f[e0 + i], p[i], mean);
  part[0][q][tok] = g * dg;
  part[1][q][tok] = mean;
  __syncthreads();
  float total = 0.f;
  mean = 0.f;
#pragma unroll
  for (int i = 0; i < kDzParts; ++i) total += part[0][i][tok], mean += part[1][i][tok];
  // The gates' terms at the selected experts.  The same expert may come twice:
  // the first of its slots adds them all, in order.
  if (a.dgate) {
    const bool use = live && sel >= 0 && sel < a.E;
    const float rest = a.gate_scale == 1.f ? total : total / a.gate_scale;
    sel_s[q][tok] = use ? sel : -1;
    term_s[q][tok] = all ? g * dg : g * (dg - rest);
    __syncthreads();
    if (use) {
      float sum = 0.f;
      bool first = true;
#pragma unroll
      for (int j = 0; j < kMaxK; ++j) {  // slots past k are -1
        const bool same = sel_s[j][tok] == sel;
        if (same && j < q) first = false;
        if (same) sum += term_s[j][tok];
      }
      if (first) z[tok][sel] = sum;
    }
  }
  __syncthreads();
  constexpr int W = (Q + 1) / 2;
  uint32_t hi2[W], mid2[W], lo2[W];  // TC: two experts' terms to a word
#pragma unroll
  for (int i = 0; i < Q; i += 2) {
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[h] = 0.f;
      if (i + h >= Q || i + h >= mine) continue;
      const float pe = p[(i + h) % Q];
      v[h] = z[tok][e0 + i + h];
      if (live && loss) v[h] = fmaf(c * pe, f[e0 + i + h] - mean, v[h]);
      if (live && all) v[h] = fmaf(-pe, total, v[h]);
    }
    if (TC) {
      const Terms x = split(v[0]), y = split(v[1]);
      hi2[i / 2] = upper_halves(x.hi, y.hi);
      mid2[i / 2] = upper_halves(x.mid, y.mid);
      lo2[i / 2] = upper_halves(x.lo, y.lo);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (i + h < Q && i + h < mine) z[tok][e0 + i + h] = v[h];
  }
  if (TC) {
    __nv_bfloat16* row = rows_s + tok * LD;
    if (Q == 8 && per == Q) {
      // Eight experts are 16 bytes of each of three 64-wide blocks.
      uint4* at = reinterpret_cast<uint4*>(row + e0);
      at[0] = make_uint4(hi2[0], hi2[1 % W], hi2[2 % W], hi2[3 % W]);
      at[8] = make_uint4(mid2[0], mid2[1 % W], mid2[2 % W], mid2[3 % W]);
      at[16] = make_uint4(lo2[0], lo2[1 % W], lo2[2 % W], lo2[3 % W]);
    } else {
      uint16_t* at = reinterpret_cast<uint16_t*>(row) + e0;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        if (i >= mine) continue;
        at[i] = static_cast<uint16_t>(hi2[i / 2] >> (i % 2 * 16));
        at[i + terms.stride] = static_cast<uint16_t>(mid2[i / 2] >> (i % 2 * 16));
        at[i + 2 * terms.stride] = static_cast<uint16_t>(lo2[i / 2] >> (i % 2 * 16));
      }
    }
  }
  __syncthreads();
  const int rows = min(kRbTokens, a.T - t0);
  if (TC) {
    const int chunks = 8 * terms.blocks;  // 16-byte chunks of a row
    uint4* out = static_cast<uint4*>(dz) + static_cast<int64_t>(t0) * chunks;
    const int ch = tid % 8;               // 8 x 32 threads: rows, then blocks
    for (int r = tid / 8; r < rows; r += kDzThreads / 8)
      for (int b = 0; b < terms.blocks; ++b)
        out[r * chunks + b * 8 + ch] =
            reinterpret_cast<const uint4*>(rows_s + r * LD)[b * 8 + ch];
  } else {
    float* out = static_cast<float*>(dz) + static_cast<int64_t>(t0) * EP;
    const int shift = __ffs(EP) - 1;      // EP is a power of two
    for (int i = tid; i < rows * EP; i += kDzThreads) {
      const int e = i & (EP - 1);
      out[i] = e < a.E ? z[i >> shift][e] : 0.f;
    }
  }
  // Column sums: 64 threads, one an expert, on each quarter of the tokens.
  const int e = tid % kMaxE, quarter = tid / kMaxE;
  float s = 0.f;
  if (e < a.E)
#pragma unroll
    for (int r = 0; r < kRbTokens / 4; ++r) s += z[quarter * (kRbTokens / 4) + r][e];
  sum_s[quarter][e] = s;
  __syncthreads();
  if (quarter == 0)
    bias_part[static_cast<int64_t>(blockIdx.x) * kMaxE + e] =
        (sum_s[0][e] + sum_s[1][e]) + (sum_s[2][e] + sum_s[3][e]);
}

// Both products of an fp32 layer, on fp32 FMA.  A CTA owns 64 columns and a
// range of tokens, in tiles of 64 tokens that cp.async brings two stages deep.
// Register tiles of 4 x 4 in both products (columns x experts over the tokens;
// tokens x columns over the experts) take two 16-byte shared-memory reads for
// 16 FMA (4096 x 1024: 8 experts 13.8 us for the pass, 7.7 at 6.56 TB/s; 64
// experts 41 us, the reads' pipe at three quarters of its rate on the busiest
// SMs; tiles of 8 x 8 and 8 x 4 on 128 columns leave one CTA an SM and took 40.5
// there, but 44.5 us against 43.3 for 2048 x 4096 with 32 experts and 21 against
// 16 for 700 x 256 with 64).  With fewer than 64 experts the threads that dW_g does not need
// share out the tile's tokens, and are added up when the range is done.
template <int EP>
struct SimtSmem {
  float x[2][kTile][kCols];
  float dz[2][kTile][EP];
  float w[EP][kCols + 4];    // W_g of the columns, expert-major; padded: a warp's
                             // stores of a column's experts would share a bank
  float4 scratch[kThreads];
  uint32_t last;
};

template <int EP>
__global__ void __launch_bounds__(kThreads, 2)
    route_products_kernel(const RouteBackwardArgs a, const RouteSums sums, int ranges, int tiles,
                          const float* __restrict__ dz) {
  constexpr int EG = EP / 4;                 // expert groups of dW_g
  constexpr int TG = kThreads / (16 * EG);   // token groups of dW_g
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<EP>& sm = *reinterpret_cast<SimtSmem<EP>*>(smem_raw);
  const float* x = static_cast<const float*>(a.x);
  const float* Wg = static_cast<const float*>(a.Wg);
  const float* dx_acc = static_cast<const float*>(a.dx_acc);
  float* dx = static_cast<float*>(a.dx);
  const int tid = threadIdx.x, cg = tid % 16, c0 = blockIdx.x * kCols;
  const int cols = min(kCols, a.d - c0);
  const bool in = 4 * cg < cols;             // columns come in eights
  const int64_t col = c0 + 4 * cg;
  // Unsigned: the end of the last tile may pass 2^31.
  const uint32_t t0 = static_cast<uint32_t>(static_cast<int64_t>(blockIdx.y) * tiles / ranges) * kTile;
  const uint32_t t1 = min(static_cast<uint32_t>(a.T),
                          static_cast<uint32_t>(static_cast<int64_t>(blockIdx.y + 1) * tiles /
                                                ranges) * kTile);
  auto load_x = [&](uint32_t tb, int st) {
    const int rows = min(static_cast<uint32_t>(kTile), t1 - tb);
    if (a.dWg)
#pragma unroll
      for (int r = tid / 16; r < kTile; r += kThreads / 16) {
        // Nothing is read of a padding token (nor past the range): zeros.
        const bool use = in && r < rows && (!a.mask || a.mask[tb + r]);
        cp_async16(smem_u32(&sm.x[st][r][4 * cg]),
                   use ? x + static_cast<int64_t>(tb + r) * a.d + col : x, use ? 16 : 0);
      }
  };
  auto load_dz = [&](uint32_t tb, int st) {
    const int rows = min(static_cast<uint32_t>(kTile), t1 - tb);
    const float* from = dz + static_cast<int64_t>(tb) * EP;
#pragma unroll
    for (int i = tid; i < kTile * EP / 4; i += kThreads) {
      const bool use = i < rows * EP / 4;
      cp_async16(smem_u32(&sm.dz[st][0][0] + 4 * i), use ? from + 4 * i : from, use ? 16 : 0);
    }
    cp_async_commit();
  };
  // The dz kernel has waited for everything before it, so the call's inputs
  // may be read before its end.
  if (t0 < t1) load_x(t0, 0);
  if (dx) {
    for (int i = tid; i < EP * (kCols + 4); i += kThreads) (&sm.w[0][0])[i] = 0.f;
    __syncthreads();
    int c = tid / a.E, e = tid % a.E;
    const int dc = kThreads / a.E, de = kThreads % a.E;
    for (int i = tid; i < cols * a.E; i += kThreads) {
      sm.w[e][c] = Wg[static_cast<int64_t>(c0) * a.E + i];
      c += dc;
      e += de;
      if (e >= a.E) e -= a.E, ++c;
    }
  }
  pdl_wait();
  pdl_trigger();
  if (t0 < t1) load_dz(t0, 0);
  const int eg = tid / 16 % EG, tg = tid / (16 * EG);
  float acc[4][4] = {};
  int st = 0;
  for (uint32_t tb = t0; tb < t1; tb += kTile, st ^= 1) {
    const int rows = min(static_cast<uint32_t>(kTile), t1 - tb);
    if (tb + kTile < t1)
      load_x(tb + kTile, st ^ 1), load_dz(tb + kTile, st ^ 1);
    else
      cp_async_commit();  // one group a tile, so that the wait counts tiles
    // This thread's four tokens and columns of dx.
    const int row = tid / 16 * 4;
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = dx_acc && dx && in && row + i < rows
                 ? *reinterpret_cast<const float4*>(
                       dx_acc + static_cast<int64_t>(tb + row + i) * a.d + col)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    cp_async_wait<1>();
    __syncthreads();
    if (a.dWg) {
#pragma unroll 4
      for (int r = tg; r < kTile; r += TG) {
        const float4 xv = *reinterpret_cast<const float4*>(&sm.x[st][r][4 * cg]);
        const float4 zv = *reinterpret_cast<const float4*>(&sm.dz[st][r][4 * eg]);
        const float xs[4] = {xv.x, xv.y, xv.z, xv.w}, zs[4] = {zv.x, zv.y, zv.z, zv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(xs[i], zs[e], acc[i][e]);
      }
    }
    if (dx) {
      float o[4][4] = {};
#pragma unroll 2
      for (int e = 0; e < EP; e += 4) {
        float zs[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 zv = *reinterpret_cast<const float4*>(&sm.dz[st][row + i][e]);
          zs[i][0] = zv.x, zs[i][1] = zv.y, zs[i][2] = zv.z, zs[i][3] = zv.w;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 wv = *reinterpret_cast<const float4*>(&sm.w[e + u][4 * cg]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i][0] = fmaf(zs[i][u], wv.x, o[i][0]);
            o[i][1] = fmaf(zs[i][u], wv.y, o[i][1]);
            o[i][2] = fmaf(zs[i][u], wv.z, o[i][2]);
            o[i][3] = fmaf(zs[i][u], wv.w, o[i][3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (in && row + i < rows)
          *reinterpret_cast<float4*>(dx + static_cast<int64_t>(tb + row + i) * a.d + col) =
              make_float4(v[i].x + o[i][0], v[i].y + o[i][1], v[i].z + o[i][2], v[i].w + o[i][3]);
    }
    __syncthreads();  // the next load goes to this stage
  }
  if (sums.dbias && tid < 32)
    for (int e = blockIdx.x + blockIdx.y * gridDim.x; e < a.E; e += gridDim.x * gridDim.y)
      sum_bias(sums, e, tid);
  if (!a.dWg) return;
  // The token groups' parts, in order, then the range's part to memory.
  // Parts [TG][64 columns][EP], 16 KB, in pieces of 16 bytes whose place is
  // xored with the column group, so that a warp's stores miss one another's
  // banks.
  float* part = &sm.x[0][0][0];
  auto place = [](int column, int e) {  // of all token groups' columns
    return ((column * EG + e / 4) ^ (column / 4 & 7)) * 4 + e % 4;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(part + place(tg * kCols + 4 * cg + i, 4 * eg)) =
        make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  __syncthreads();
  {
    float* out = sums.dw + (static_cast<int64_t>(blockIdx.y) * a.d + c0) * a.E;
    int c = tid / a.E, e = tid % a.E;
    const int dc = kThreads / a.E, de = kThreads % a.E;
    for (int i = tid; i < cols * a.E; i += kThreads) {
      float sum = part[place(c, e)];
#pragma unroll
      for (int g = 1; g < TG; ++g) sum += part[place(g * kCols + c, e)];
      out[i] = sum;
      c += dc;
      e += de;
      if (e >= a.E) e -= a.E, ++c;
    }
  }
  if (sums.many) return;
  __threadfence();
  __syncthreads();
  if (tid == 0)
    sm.last = atomicAdd(sums.tickets + blockIdx.x, 1u) + 1 == static_cast<uint32_t>(ranges);
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  sum_ranges(sums, c0, cols, tid, kThreads, sm.scratch, [] { __syncthreads(); });
}

// dW_g from many ranges' parts: 32 pieces of 16 bytes a CTA, each by eight
// warps that share out the ranges and are added up in order.
__global__ void __launch_bounds__(kThreads) route_finish_kernel(const RouteSums s) {
  constexpr int G = kThreads / 32;
  __shared__ float4 part[G][32];
  const int lane = threadIdx.x % 32, g = threadIdx.x / 32;
  const int64_t n = static_cast<int64_t>(s.d) * s.E / 4;  // columns come in eights
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  pdl_wait();
  pdl_trigger();
  const float4* from = reinterpret_cast<const float4*>(s.dw) + v;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& b) { sum.x += b.x, sum.y += b.y, sum.z += b.z, sum.w += b.w; };
  if (v < n)
#pragma unroll 8
    for (int r = g; r < s.ranges; r += G) add(from[r * n]);
  part[g][lane] = sum;
  __syncthreads();
  if (g > 0 || v >= n) return;
  for (int i = 1; i < G; ++i) add(part[i][lane]);
  if (*s.err != 0) sum.x = sum.y = sum.z = sum.w = __int_as_float(0x7fc00000);
  reinterpret_cast<float4*>(s.dWg)[v] = sum;
}

// The bias alone: one warp an expert.
__global__ void __launch_bounds__(32) route_bias_kernel(const RouteSums sums) {
  pdl_wait();
  pdl_trigger();
  sum_bias(sums, blockIdx.x, threadIdx.x);
}

cudaError_t launch_products(const RouteBackwardArgs& a, const RouteBackwardPlan& p,
                            const RouteSums& sums, const float* dz, cudaStream_t s) {
  auto go = [&](auto kern, size_t smem) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(p.cols, p.ranges), dim3(kThreads), smem, s, 1, true, a, sums,
                         p.ranges, p.tiles, dz);
  };
  switch (p.EP) {
    case 8: return go(route_products_kernel<8>, sizeof(SimtSmem<8>));
    case 16: return go(route_products_kernel<16>, sizeof(SimtSmem<16>));
    case 32: return go(route_products_kernel<32>, sizeof(SimtSmem<32>));
    default: return go(route_products_kernel<64>, sizeof(SimtSmem<64>));
  }
}

}  // namespace

size_t route_backward_scratch_bytes(int T, int d, int E, moe_dtype dtype) {
  return make_plan(T, d, E, dtype).total;
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, moe_dtype dtype, cudaStream_t s) {
  if (a.T == 0) {
    cudaError_t err = cudaSuccess;
    if (a.dWg) err = cudaMemsetAsync(a.dWg, 0, sizeof(float) * a.d * a.E, s);
    if (a.dbias && err == cudaSuccess) err = cudaMemsetAsync(a.dbias, 0, sizeof(float) * a.E, s);
    return err;
  }
  const RouteBackwardPlan p = make_plan(a.T, a.d, a.E, dtype);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  float* bias = reinterpret_cast<float*>(ws + p.bias);
  const RouteSums sums{bias,
                       reinterpret_cast<float*>(ws + p.dw),
                       reinterpret_cast<int32_t*>(ws + p.err),
                       reinterpret_cast<uint32_t*>(ws + p.tickets),
                       a.dWg,
                       a.dbias,
                       p.blocks,
                       p.ranges,
                       a.d,
                       a.E,
                       p.many};
  if (route_backward_is_small(a.T, a.d, a.E))
    return launch_route_backward_small(a, dtype, sums.err, s);
  const bool tc = dtype == MOE_BF16;
  auto dz = [&](auto kern) {
    return launch_kernel(kern, dim3(p.blocks), dim3(kDzThreads), 0, s, 1, true, a, p.EP,
                         dz_terms(a.E), static_cast<void*>(ws + p.dz), bias, sums.err,
                         sums.tickets, p.cols);
  };
  cudaError_t err =
      a.E <= 8    ? (tc ? dz(route_dz_kernel<true, 1>) : dz(route_dz_kernel<false, 1>))
      : a.E <= 16 ? (tc ? dz(route_dz_kernel<true, 2>) : dz(route_dz_kernel<false, 2>))
      : a.E <= 32 ? (tc ? dz(route_dz_kernel<true, 4>) : dz(route_dz_kernel<false, 4>))
                  : (tc ? dz(route_dz_kernel<true, 8>) : dz(route_dz_kernel<false, 8>));
  if (err != cudaSuccess) return err;
  if (!a.dx && !a.dWg) return launch_kernel(route_bias_kernel, dim3(a.E), dim3(32), 0, s, 1, true, sums);
  err = tc ? launch_route_products_tc(a, p, sums, s)
           : launch_products(a, p, sums, reinterpret_cast<const float*>(ws + p.dz), s);
  if (err != cudaSuccess || !a.dWg || !sums.many) return err;
  const int64_t pieces = static_cast<int64_t>(a.d) * a.E / 4;
  return launch_kernel(route_finish_kernel, dim3(static_cast<unsigned>((pieces + 31) / 32)),
                       dim3(kThreads), 0, s, 1, true, sums);
}

}  // namespace moe
