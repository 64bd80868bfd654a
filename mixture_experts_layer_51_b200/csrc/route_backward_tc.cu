// The two products of the router's backward pass for bf16 layers, on the
// tensor cores, in one pass over x:
//
//     dW_g = x^T dz   (M = 128 columns, N = experts x terms, K = tokens)
//     dx = dx_acc + dz W_g^T   (M = 128 tokens, N = 128 columns, K = experts)
//
// A CTA owns 128 columns and a range of tokens, in tiles of 128 tokens.  Per
// tile TMA brings 128 x 128 of x and the tokens' dz terms (route_backward.cuh)
// into one stage of a ring; the same dz bytes are the N-major operand of the
// first product and the K-major operand of the second.  dW_g accumulates in
// tensor memory over the whole range; dx of a tile goes through one of two
// accumulators to the epilogue warps, which add dx_acc (brought by TMA into
// the buffer that the result leaves from), round once and store by TMA.
// Bound by HBM: x is read once and dx written once; dz is re-read from L2 by
// every column block.
//
// Warps: 0 TMA loads, 1 MMA issue, 2 TMA stores (and the loads of dx_acc), 3
// zeroes the rows of padding tokens in x (with a mask only: their x may hold
// anything, and 0 * NaN is NaN), 4-11 epilogue, in two groups that take the
// 64-column halves of the tiles in turn.  Every wait is bounded; a time-out
// raises the workspace's error word and the CTA leaves after its copies and
// MMAs have landed, its block of dx (and its columns of dW_g) filled with NaN.
//
// Measured on one B200, all launches of the backward pass (floors at
// 6.56 TB/s in brackets): 8192 x 4096, 8 experts, with dx_acc 40.0 us (30.8),
// without 29.5 (20.6); 16384 x 2048 without dx_acc: 32 experts 37.1 us, 64
// experts 40.2 (21.3), 41.5 with a mask that leaves out one token in six.  A
// tile takes 1.5 us there, of which its 64 KB take 1.45 at the HBM rate of 144
// CTAs (with dz in two terms in dx's product instead of three, the masked pass
// took 39.9; dx then was off by 2^-17 of its terms where they cancel);
// the rest is the dz kernel (7 us, which the first tiles' x is loaded behind)
// and about 7 us of start, last tile and sums.  On fp32 FMA the same passes
// took 181 and 778 us.  A second epilogue group and stores from a warp of
// their own took the products of the first shape from 47 to 34 us; laying W_g
// out element by element from memory had cost 4 us of every launch.

#include <cudaTypedefs.h>

#include <stdlib.h>

#include <atomic>
#include <mutex>

#include "route_backward.cuh"

namespace moe {
namespace {

constexpr int kEpilogue = 256;        // threads of warps 4-11
constexpr int kThreads = 128 + kEpilogue;
constexpr int kUnit = 128 * 64 * 2;   // 64 columns (or experts) of 128 rows: 16 KB
constexpr int kMaxStages = 3;
constexpr int kMaxUnits = 4;
constexpr int kDwCol = 256;           // dW_g's first column in tensor memory
// Tiles whose products the tensor cores sum up before the epilogue moves the
// sum into fp32 registers.  The accumulators in tensor memory do not round
// to nearest: over a whole range (16 tiles) dW_g came out 2.5e-6 off, twice
// to ten times what sums that round are off.
constexpr int kFlush = 4;
constexpr int kSmem = 14 * kUnit + 2048;  // + control block and alignment
constexpr int kPartBytes = kRbPartBytes;
static_assert(kPartBytes == kEpilogue * 32 * 4, "32 floats a thread");

// NB: 64-element blocks of a dz row.  Stages x (2 + NB), W_g blocks and
// staging units add up to the same 14 blocks of shared memory.
template <int NB>
struct Cfg {
  static constexpr int STAGES = NB == 1 ? 3 : 2;
  static constexpr int WB = NB == 3 ? 1 : NB;
  static constexpr int UNITS = NB == 3 ? 3 : 4;
  static constexpr int STAGE = (2 + NB) * kUnit;
  static constexpr int W_OFF = STAGES * STAGE;
  static constexpr int OUT_OFF = W_OFF + WB * kUnit;
  static constexpr int CTL_OFF = OUT_OFF + UNITS * kUnit;
};
static_assert(Cfg<1>::CTL_OFF == 14 * kUnit && Cfg<2>::CTL_OFF == 14 * kUnit &&
              Cfg<3>::CTL_OFF == 14 * kUnit, "one shared-memory size");

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages], clean[kMaxStages];
  uint64_t tfull[2], tempty[2];                    // dx accumulators
  uint64_t uready[kMaxUnits], ustaged[kMaxUnits];  // staging units
  uint64_t dwfull, dwempty, wready, drain, never;
  uint32_t tmem_base;
  uint32_t last;  // this CTA finished last of its column block
  volatile int abort_flag;
};

struct Params {
  const __nv_bfloat16* Wg;
  const uint8_t* mask;
  __nv_bfloat16* dx;  // what a CTA that gave up marks; the results leave by TMA
  RouteSums sums;
  int T, d, E, stride, cols, ranges, tiles;
  int want_dx, want_dw, add;
  int debug_stall;  // 1: CTA 0's MMA issuer first waits on a barrier nobody arms (tests only)
};

__device__ __forceinline__ void give_up(const Params& p, Ctl& c, int code) {
  if (!c.abort_flag) atomicOr(p.sums.err, code);
  c.abort_flag = 1;
}

// Byte offset of 16-byte chunk `ch` of row r in a 128-byte-swizzled block.
__device__ __forceinline__ uint32_t swz(int r, int ch) {
  return static_cast<uint32_t>(r * 128 + ((ch ^ (r & 7)) << 4));
}

__device__ __forceinline__ void epilogue_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kEpilogue) : "memory");
}
// The same, and whether all threads say so: one answer for all of them.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, 1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(ok)), "n"(kEpilogue)
      : "memory");
  return all != 0;
}

template <int NB>
__global__ void __launch_bounds__(kThreads, 1)
    route_products_tc_kernel(const __grid_constant__ CUtensorMap tmX,
                             const __grid_constant__ CUtensorMap tmDz,
                             const __grid_constant__ CUtensorMap tmAcc,
                             const __grid_constant__ CUtensorMap tmDx, const Params p) {
  using C = Cfg<NB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctl& c = *reinterpret_cast<Ctl*>(smem + C::CTL_OFF);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = static_cast<int>(blockIdx.x % p.cols) * kRbTcCols;
  const int range = blockIdx.x / p.cols;
  const int tile0 = static_cast<int>(static_cast<int64_t>(range) * p.tiles / p.ranges);
  const int ntiles =
      static_cast<int>(static_cast<int64_t>(range + 1) * p.tiles / p.ranges) - tile0;
  const int halves = c0 + 64 < p.d ? 2 : 1;  // 64-column halves that exist
  const int units = p.want_dx ? ntiles * halves : 0;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(smem_u32(&c.full[i]), 1);
      mbar_init(smem_u32(&c.empty[i]), 1);
      mbar_init(smem_u32(&c.clean[i]), 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&c.tfull[i]), 1);
      mbar_init(smem_u32(&c.tempty[i]), 4 * halves);
    }
    for (int i = 0; i < C::UNITS; ++i) {
      mbar_init(smem_u32(&c.uready[i]), 1);
      mbar_init(smem_u32(&c.ustaged[i]), 128);
    }
    mbar_init(smem_u32(&c.dwfull), 1);
    mbar_init(smem_u32(&c.dwempty), kEpilogue / 32);
    mbar_init(smem_u32(&c.wready), kEpilogue);
    mbar_init(smem_u32(&c.drain), 1);
    mbar_init(smem_u32(&c.never), 1);
    c.abort_flag = 0;
    fence_mbar_init();
    fence_async_shared();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&c.tmem_base), 512);
    tmem_relinquish();
  }
  if (tid == 64) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmDz);
    tma_prefetch_desc(&tmAcc);
    tma_prefetch_desc(&tmDx);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  // This kernel may start once every CTA of the dz kernel is past its own
  // pdl_wait, so all that came before that one is done: x, W_g and dx_acc are
  // read at once, and only what the dz kernel writes waits for its end.
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------ TMA loads
      const int nx = p.want_dw ? halves : 0;
      auto load_x = [&](int i, int stage) {
        const uint32_t bar = smem_u32(&c.full[stage]);
        mbar_arrive_expect_tx(bar, (nx + NB) * kUnit);
        for (int h = 0; h < nx; ++h)
          tma_load_2d(base + stage * C::STAGE + h * kUnit, &tmX, bar, c0 + 64 * h,
                      (tile0 + i) * kRbTcTokens);
      };
      const int early = min(C::STAGES, ntiles);
      for (int i = 0; i < early; ++i) load_x(i, i);
      pdl_wait();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int i = 0; i < ntiles; ++i) {
        if (i >= early) {
          if (c.abort_flag || !mbar_wait(smem_u32(&c.empty[stage]), phase ^ 1)) {
            give_up(p, c, kErrTimeoutProducer);
            break;
          }
          load_x(i, stage);
        }
        for (int b = 0; b < NB; ++b)
          tma_load_2d(base + stage * C::STAGE + (2 + b) * kUnit, &tmDz, smem_u32(&c.full[stage]),
                      64 * b, (tile0 + i) * kRbTcTokens);
        ++issued;
        if (++stage == C::STAGES) stage = 0, phase ^= 1;
      }
      // Nothing may land after the CTA has left: stage s was filled
      // (issued - 1 - s) / STAGES + 1 times.
      for (int s = 0; s < C::STAGES && s < issued; ++s)
        if (!mbar_wait(smem_u32(&c.full[s]), ((issued - 1 - s) / C::STAGES) & 1u))
          give_up(p, c, kErrTimeoutDrain);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------ MMA issue
      constexpr uint32_t idesc_dw = idesc_bf16_f32(128, 64 * NB, true, true);
      constexpr uint32_t idesc_dx = idesc_bf16_f32(128, 128, false, false);
      const uint64_t wdesc = smem_desc_sw128(base + C::W_OFF, 16, 1024);
      bool ok = mbar_wait(smem_u32(&c.wready), 0);
      if (p.debug_stall && blockIdx.x == 0) ok = mbar_wait(smem_u32(&c.never), 0);
      if (!ok) give_up(p, c, kErrTimeoutMma);
      int stage = 0, flushed = 0;
      uint32_t phase = 0;
      for (int i = 0; ok && i < ntiles; ++i) {
        const int buf = i & 1;
        ok = !c.abort_flag &&
             mbar_wait(smem_u32(&c.full[stage]), phase) &&
             (!p.want_dx || mbar_wait(smem_u32(&c.tempty[buf]), ((i >> 1) & 1) ^ 1));
        if (!ok) {
          give_up(p, c, kErrTimeoutMma);
          break;
        }
        tc_fence_after();
        const uint32_t src = base + stage * C::STAGE;
        if (p.want_dx) {
          // 16 experts are 32 bytes of a 128-byte row.
          const uint64_t adesc = smem_desc_sw128(src + 2 * kUnit, 16, 1024);
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_bf16(tmem + buf * 128,
                          adesc + static_cast<uint64_t>((b * kUnit + kk * 32) >> 4),
                          wdesc + static_cast<uint64_t>(((b % C::WB) * kUnit + kk * 32) >> 4),
                          idesc_dx, (b > 0 || kk > 0) ? 1u : 0u);
          tc_commit(smem_u32(&c.tfull[buf]));
        }
        if (p.want_dw) {
          const bool first = i % kFlush == 0;
          if ((first && i > 0 && !mbar_wait(smem_u32(&c.dwempty), (flushed++) & 1)) ||
              (p.mask && !mbar_wait(smem_u32(&c.clean[stage]), phase))) {
            give_up(p, c, kErrTimeoutMma);
            break;
          }
          tc_fence_after();
          // 16 tokens are 16 rows of 128 bytes; 64-wide blocks lie 16 KB apart.
          const uint64_t adesc = smem_desc_sw128(src, kUnit, 1024);
          const uint64_t bdesc = smem_desc_sw128(src + 2 * kUnit, kUnit, 1024);
#pragma unroll
          for (int kk = 0; kk < kRbTcTokens / 16; ++kk)
            tc_mma_bf16(tmem + kDwCol, adesc + static_cast<uint64_t>((kk * 2048) >> 4),
                        bdesc + static_cast<uint64_t>((kk * 2048) >> 4), idesc_dw,
                        (!first || kk > 0) ? 1u : 0u);
          if (i % kFlush == kFlush - 1 || i == ntiles - 1) tc_commit(smem_u32(&c.dwfull));
        }
        tc_commit(smem_u32(&c.empty[stage]));
        if (++stage == C::STAGES) stage = 0, phase ^= 1;
      }
      // Every MMA has completed before tensor memory is freed.
      tc_commit(smem_u32(&c.drain));
      if (!mbar_wait(smem_u32(&c.drain), 0)) give_up(p, c, kErrTimeoutDrain);
    }
  } else if (warp == 2) {
    if (lane == 0) {
      // ---------------------------------------- staging units and stores
      // A unit is ready when its last store has left and, with dx_acc, the
      // tile's part of that has arrived.
      auto make_ready = [&](int u) {
        const uint32_t bar = smem_u32(&c.uready[u % C::UNITS]);
        if (!p.add) {
          mbar_arrive(bar);
          return;
        }
        mbar_arrive_expect_tx(bar, kUnit);
        tma_load_2d(base + C::OUT_OFF + (u % C::UNITS) * kUnit, &tmAcc, bar,
                    c0 + 64 * (u % halves), (tile0 + u / halves) * kRbTcTokens);
      };
      int readied = 0;
      // The epilogue lays W_g out by way of the first unit.
      const bool laid = mbar_wait(smem_u32(&c.wready), 0);
      if (!laid) give_up(p, c, kErrTimeoutEpilogue);
      for (; laid && readied < C::UNITS && readied < units; ++readied) make_ready(readied);
      for (int u = 0; u < units; ++u) {
        const int slot = u % C::UNITS;
        if (c.abort_flag || !mbar_wait(smem_u32(&c.ustaged[slot]), (u / C::UNITS) & 1)) {
          give_up(p, c, kErrTimeoutEpilogue);
          break;
        }
        tma_store_2d(&tmDx, base + C::OUT_OFF + slot * kUnit, c0 + 64 * (u % halves),
                     (tile0 + u / halves) * kRbTcTokens);
        bulk_commit();
        // The unit before has left its place by now, or nearly.
        if (u > 0 && readied < units) {
          bulk_wait_read<1>();
          make_ready(readied++);
        }
      }
      bulk_wait<0>();
      // No load of dx_acc may land after the CTA has left.
      for (int u = readied > C::UNITS ? readied - C::UNITS : 0; u < readied; ++u)
        if (!mbar_wait(smem_u32(&c.uready[u % C::UNITS]), (u / C::UNITS) & 1))
          give_up(p, c, kErrTimeoutDrain);
    }
  } else if (warp == 3) {
    // --------------------------------------------- rows of padding tokens
    int stage = 0;
    uint32_t phase = 0;
    // Bit r of lane l's word q: row 32 q + l of the tile is padding.
    auto padding = [&](int i) {
      uint32_t bits = 0;
      for (int q = 0; q < 4; ++q) {
        const int t = (tile0 + i) * kRbTcTokens + 32 * q + lane;
        if (t < p.T && !p.mask[t]) bits |= 1u << q;
      }
      return bits;
    };
    // Without dW_g nobody reads x, and nobody waits for `clean`: following the
    // ring then would be a wait that the ring could overtake.
    const bool scrub = p.mask && p.want_dw;
    uint32_t bits = scrub ? padding(0) : 0;
    for (int i = 0; scrub && i < ntiles; ++i) {
      const uint32_t next = i + 1 < ntiles ? padding(i + 1) : 0;
      if (!__all_sync(0xffffffffu, !c.abort_flag && mbar_wait(smem_u32(&c.full[stage]), phase))) {
        give_up(p, c, kErrTimeoutMma);
        break;
      }
      // Four rows a step, 16 bytes of each half a lane: the same time for one
      // padding token as for a tile of them.
      uint8_t* x = smem + stage * C::STAGE + lane * 16;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t rows = __ballot_sync(0xffffffffu, (bits >> q) & 1u);
        if (!rows) continue;
#pragma unroll
        for (int g = 0; g < 8; ++g)
          if (rows >> (4 * g + lane / 8) & 1u) {
            const int at = (32 * q + 4 * g) * 128;
            *reinterpret_cast<uint4*>(x + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(x + kUnit + at) = make_uint4(0, 0, 0, 0);
          }
      }
      fence_async_shared();
      mbar_arrive(smem_u32(&c.clean[stage]));
      bits = next;
      if (++stage == C::STAGES) stage = 0, phase ^= 1;
    }
    if (p.sums.dbias) {
      pdl_wait();
      for (int e = blockIdx.x; e < p.E; e += gridDim.x) sum_bias(p.sums, e, lane);
    }
  } else {
    // --------------------------------------------------------- epilogue
    const int et = tid - 128, group = et >> 7, q = warp & 3, row = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    if (p.want_dx) {
      // W_g of the block as the K-major operand: term after term, zero past
      // the last expert and column.  The block's rows are contiguous, so they
      // come in 16-byte pieces into the first staging unit (dx_acc waits for
      // wready) and are spread out from there.
      uint8_t* raw = smem + C::OUT_OFF;
      const int bytes = min(kRbTcCols, p.d - c0) * p.E * 2;  // columns come in eights
      const uint8_t* from = reinterpret_cast<const uint8_t*>(p.Wg + static_cast<int64_t>(c0) * p.E);
      for (int i = et * 16; i < kUnit; i += kEpilogue * 16)
        *reinterpret_cast<uint4*>(raw + i) =
            i < bytes ? *reinterpret_cast<const uint4*>(from + i) : make_uint4(0, 0, 0, 0);
      epilogue_sync();
      const uint16_t* w = reinterpret_cast<const uint16_t*>(raw);
#pragma unroll
      for (int j = 0; j < 4 * C::WB; ++j) {
        const int i = et + j * kEpilogue, r = i / (8 * C::WB), n = i % (8 * C::WB);
        int e = NB == 3 ? 8 * n : 8 * n % p.stride;
        int left = (NB == 3 ? p.E : 3 * p.stride) - 8 * n;  // elements that are not zero
        uint32_t v[4];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t x = left > u ? w[r * p.E + e] : 0u;
          v[u / 2] = u % 2 ? v[u / 2] | (x << 16) : x;
          if (++e == p.stride) e = 0;
        }
        *reinterpret_cast<uint4*>(smem + C::W_OFF + n / 8 * kUnit + swz(r, n % 8)) =
            make_uint4(v[0], v[1], v[2], v[3]);
      }
      fence_async_shared();
    }
    mbar_arrive(smem_u32(&c.wready));
    // dW_g so far: lane = column; 32 NB of the block's columns a thread, the
    // three terms of one expert already added where their places are known.
    constexpr int ACC = NB == 3 ? 32 : 32 * NB;
    float acc[ACC];
#pragma unroll
    for (int e = 0; e < ACC; ++e) acc[e] = 0.f;
    int u = group, flushes = 0;
    bool ok = true;
    for (int i = 0; i < ntiles && ok; ++i) {
      for (; ok && u < units && u / halves == i; u += 2) {
        const int buf = i & 1, slot = u % C::UNITS;
        ok = __all_sync(0xffffffffu,
                        !c.abort_flag && mbar_wait(smem_u32(&c.tfull[buf]), (i >> 1) & 1) &&
                            mbar_wait(smem_u32(&c.uready[slot]), (u / C::UNITS) & 1));
        if (!ok) break;
        tc_fence_after();
        float v[2][32];
        const uint32_t src = tmem + lane_base + buf * 128 + u % halves * 64;
        tc_ld_32cols(src, v[0]);
        tc_ld_32cols(src + 32, v[1]);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.tempty[buf]));
        uint8_t* out = smem + C::OUT_OFF + slot * kUnit;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          uint4* at = reinterpret_cast<uint4*>(out + swz(row, ch));
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = v[ch / 4][ch % 4 * 8 + e];
          if (p.add) {
            const uint4 a = *at;
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[2 * e] += __uint_as_float(w[e] << 16);
              f[2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
            }
          }
          *at = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                           pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        }
        fence_async_shared();
        mbar_arrive(smem_u32(&c.ustaged[slot]));
      }
      if (ok && p.want_dw && (i % kFlush == kFlush - 1 || i == ntiles - 1)) {
        ok = __all_sync(0xffffffffu,
                        !c.abort_flag && mbar_wait(smem_u32(&c.dwfull), (flushes++) & 1));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float v[32];
          tc_ld_32cols(tmem + lane_base + kDwCol +
                           (NB == 3 ? (2 - b) * 64 + group * 32 : (group * NB + b) * 32), v);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[(NB == 3 ? 0 : b * 32) + e] += v[e];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.dwempty));
      }
    }
    if (!ok) give_up(p, c, kErrTimeoutEpilogue);
    if (p.want_dw) {
      ok = epilogue_all(ok);
      const int block = blockIdx.x % p.cols, ncols = min(kRbTcCols, p.d - c0), n = ncols * p.E;
      // The block's rows go through the ring, which is idle after the last
      // flush, so that they leave in whole lines: f(i, value) for element i of
      // [columns][E].
      constexpr int LD = 2 * ACC + 1;
      float* rows = reinterpret_cast<float*>(smem);
      auto through_ring = [&](auto f) {
#pragma unroll
        for (int e = 0; e < ACC; ++e) rows[row * LD + group * ACC + e] = acc[e];
        epilogue_sync();
        int r = et / p.E, e = et % p.E;
        const int dr = kEpilogue / p.E, de = kEpilogue % p.E;
        for (int i = et; i < n; i += kEpilogue) {
          const float* at = rows + r * LD + e;
          f(i, NB == 3 ? at[0] : at[2 * p.stride] + at[p.stride] + at[0]);
          r += dr;
          e += de;
          if (e >= p.E) e -= p.E, ++r;
        }
      };
      // A range's part: three blocks of terms are already one value an
      // expert, so the registers leave as they are, 16 bytes a thread; with
      // fewer, the terms are added first.
      float4* mine = reinterpret_cast<float4*>(p.sums.dw) + block * (kPartBytes / 16) + et;
      const int64_t plane = static_cast<int64_t>(p.cols) * (kPartBytes / 16);
      const bool as_held = NB == 3 && !p.sums.many;
      if (ok && as_held) {
#pragma unroll
        for (int j = 0; j < ACC / 4; ++j)
          mine[range * plane + j * kEpilogue] =
              make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
      } else if (ok) {
        float* out = p.sums.dw + (static_cast<int64_t>(range) * p.d + c0) * p.E;
        through_ring([&](int i, float v) { out[i] = v; });
      }
      bool last = false;
      if (!p.sums.many) {
        __threadfence();
        epilogue_sync();
        if (et == 0)
          c.last = atomicAdd(p.sums.tickets + block, 1u) + 1 == static_cast<uint32_t>(p.ranges);
        epilogue_sync();
        last = c.last;
      }
      if (last) {
        __threadfence();
        if (NB == 3) {
          const bool failed = *static_cast<volatile int32_t*>(p.sums.err) != 0;
          float own[ACC];
#pragma unroll
          for (int e = 0; e < ACC; ++e) own[e] = acc[e], acc[e] = 0.f;
#pragma unroll 2
          for (int r = 0; r < p.ranges; ++r) {
#pragma unroll
            for (int j = 0; j < ACC / 4; ++j) {
              const float4 v = r == range ? make_float4(own[4 * j], own[4 * j + 1], own[4 * j + 2],
                                                        own[4 * j + 3])
                                          : __ldcg(mine + r * plane + j * kEpilogue);
              acc[4 * j] += v.x, acc[4 * j + 1] += v.y, acc[4 * j + 2] += v.z,
                  acc[4 * j + 3] += v.w;
            }
          }
          float* out = p.sums.dWg + static_cast<int64_t>(c0) * p.E;
          through_ring(
              [&](int i, float v) { out[i] = failed ? __int_as_float(0x7fc00000) : v; });
        } else {
          sum_ranges(p.sums, c0, ncols, et, kEpilogue, reinterpret_cast<float4*>(smem),
                     epilogue_sync);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (c.abort_flag && p.want_dx) {
    // Which tiles were stored is not known here: none of them counts.
    const int chunks = min(kRbTcCols, p.d - c0) / 8;  // columns come in eights
    const int rows = min(ntiles * kRbTcTokens, p.T - tile0 * kRbTcTokens);
    __nv_bfloat16* to = p.dx + static_cast<int64_t>(tile0) * kRbTcTokens * p.d + c0;
    const uint4 nan = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    for (int64_t i = tid; i < static_cast<int64_t>(rows) * chunks; i += kThreads)
      *reinterpret_cast<uint4*>(to + i / chunks * p.d + i % chunks * 8) = nan;
  }
}

// Failure-detection tests: MOE_DEBUG_STALL_ROUTE=N lets one CTA of the next N
// launches run out of its waits (read once per process).
int take_debug_stall() {
  static std::atomic<int> budget{[] {
    const char* v = getenv("MOE_DEBUG_STALL_ROUTE");
    return v ? atoi(v) : 0;
  }()};
  int cur = budget.load();
  while (cur > 0 && !budget.compare_exchange_weak(cur, cur - 1)) {
  }
  return cur > 0 ? 1 : 0;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// bf16 [rows, cols], boxes of 64 columns x 128 rows, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* at, uint64_t rows, uint64_t cols) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, 128};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(at), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_route_products_tc(const RouteBackwardArgs& a, const RouteBackwardPlan& p,
                                     const RouteSums& sums, cudaStream_t s) {
  const DzTerms t = dz_terms(a.E);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  CUtensorMap mx, mdz, macc, mdx;
  // A map that the call does not use is a copy of dz's.
  if (!make_map(&mdz, ws + p.dz, a.T, 64 * t.blocks)) return cudaErrorInvalidValue;
  mx = macc = mdx = mdz;
  if ((a.dWg && !make_map(&mx, a.x, a.T, a.d)) || (a.dx && !make_map(&mdx, a.dx, a.T, a.d)) ||
      (a.dx && a.dx_acc && !make_map(&macc, a.dx_acc, a.T, a.d)))
    return cudaErrorInvalidValue;
  Params k{static_cast<const __nv_bfloat16*>(a.Wg),
           a.mask,
           static_cast<__nv_bfloat16*>(a.dx),
           sums,
           a.T,
           a.d,
           a.E,
           t.stride,
           p.cols,
           p.ranges,
           p.tiles,
           a.dx != nullptr,
           a.dWg != nullptr,
           a.dx && a.dx_acc,
           take_debug_stall()};
  auto go = [&](auto kern) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(p.cols * p.ranges), dim3(kThreads), kSmem, s, 1, true, mx, mdz,
                         macc, mdx, k);
  };
  if (t.blocks == 1) return go(route_products_tc_kernel<1>);
  if (t.blocks == 2) return go(route_products_tc_kernel<2>);
  return go(route_products_tc_kernel<3>);
}

}  // namespace moe
