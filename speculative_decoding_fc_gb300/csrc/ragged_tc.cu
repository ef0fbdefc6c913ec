// Attention over ragged key/value caches on the 5th-generation tensor cores, for groups of
// more than 16 query rows per kv head.  Schedule and masks: ragged.cuh.
//
// A CTA has two halves of 128 query rows (the MMA's M), in one of two forms:
//   shared   a row tile of 256 rows, 128 to each half, both reading every key tile (64
//            keys): the products bound the time (long queries, a batch over its prefix);
//   streams  a row tile of 64 rows (the MMA's other rows hold whatever lies behind them);
//            each half is a range of the schedule of its own, with its own keys: the reading
//            of the keys bounds the time (draft blocks), and the two keep it going while the
//            other computes or changes to another item.
// One CTA per SM, 12 warps:
//   warps 0-3, 4-7  the softmax of one half each, one thread per row;
//   warps 8, 11     TMA loads of key and value tiles into a ring of ten 16 KB stages (shared:
//                   warp 8; streams: one warp and five stages per half, and Q, in two buffers:
//                   an item's Q comes while the one before is still computed, which took up to
//                   17 thousand cycles of an item of the draft block's otherwise);
//   warps 9, 10     issue one half's MMAs each: S = Q K^T (both from shared memory, 128-byte
//                   swizzle), O += P V (P from tensor memory, V as its N-major operand: the
//                   tile is used as it was loaded, nothing is transposed).
// Tensor memory (512 columns): per half S (64 fp32 columns), two buffers of P (64 bf16, 32
// columns each; streams: P's two parts) and O (128).  Q K^T of tile t + 1 runs as soon as the
// softmax has read S of tile t, P V of tile t when its weights are there, so the tensor pipe has
// work while the softmax computes.  (With tiles of 128 keys S filled its half's columns, P had
// to take its place, and products and softmax of a half took turns: 3500 cycles per 128 keys
// of both halves, of which the pipe worked 2050.)
// Measured: 1536 rows of 40 heads over a prefix of 32749 keys, 1.03 TFLOP in 731 us: 1.41
// PFLOP/s, 72% of the bf16 peak measured with a large library product; 1710 cycles per 64
// keys of both halves (counts of cycles: clock64 in builds made for it).  Products take 1024
// of them, at 128 bytes a cycle the shared-memory reads of Q and K (48 KB for each half's 256
// cycles of Q K^T) hold the pipe about 256 longer, and a softmax takes about 1100; over a
// prefix of 16384 the pipe is active 56% of the time.  What bounds it is neither alone but the
// way between them (barriers, tensor memory, the MMA warps' own loop).  Tried and slower: a lock that keeps one half's MMAs together, half 0's Q
// in tensor memory with one buffer of P, four warpgroups of softmax with two threads a row,
// the ring's stages given back by the softmax warps instead of a commit each.
// The output is rescaled only when a row's maximum has grown by more than 2^8 since the
// last time (weights up to 2^8 lose nothing in fp32 sums or bf16 weights), which after the
// first tiles is rare.  The weights' sum is taken in fp32, before they are rounded.
// Streams form: the weights enter P V as bf16 parts hi + lo (2^-16 relative), as in the decode
// kernel and the backbone's attention, so that the same block gets the same bits of accuracy
// through any of them.  The second product's 256 cycles a tile are free where the keys'
// reading is the bound; the parts take both of P's buffers, so a tile's weights wait for the
// product before (draft block over 1032 keys 11.6 -> 12.0 us, 4 tokens over a prefix of
// 4096 15.7 -> 16.5).
// Shared form: rounded to bf16 once (half a step, 2^-8 relative, each rounding its own way: an
// output's error grows from 0.0017 to 0.0018 relative, most of it the output's own rounding).
// With two parts a prompt of 2 x 4099 tokens took 394 us for 334, 32 x 8 queries over a
// prefix of 16384 115 for 99, and 192 x 8 over 32749 1140 for 900.
// Value rows of keys that no row of the item sees are left out of P V in steps of 16 keys;
// those in a step with seen keys are zeroed in shared memory first (their weights are
// zero, but they may hold NaN or infinities).
// Waits are bounded as in gemm_tcgen05.cu.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "ragged.cuh"
#include "ragged_host.h"
#include "tcgen05.cuh"

namespace dspark {
namespace ragged {

using namespace tc;

struct TcParams {
  Args a;
  CUtensorMap k, v, kp, vp;
  CUtensorMap q, qp;   // streams form: a group's rows of q (of a request, of the prefix)
};

namespace {

constexpr int kKT = kTcKeys;
constexpr int kThreads = 384;
constexpr uint32_t kHalfTile = kKT * 128;          // [64 keys][64 dims] bf16
constexpr uint32_t kTileBytes = 2 * kHalfTile;
constexpr int kStages = 10;
// Q: [2 x 64 dims][256 rows][128 bytes]; shared form: 128 rows per half; streams form: 64 rows
// per half and buffer (the MMAs read 128, whatever they hold)
constexpr uint32_t kQHalf = 256 * 128, kQBytes = 2 * kQHalf;
constexpr uint32_t kSmem = 1024 + kQBytes + kStages * kTileBytes + 512;
constexpr float kRescale = 8.0f;                   // log2 units

// D fp32, A and B bf16, M = 128; Q K^T: N = 64; P V: N = 128, bit 16: B is N-major
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kKT >> 3) << 17) | (8u << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (16u << 17) | (8u << 24);

// Shared-memory descriptors in two words.  The low one: address / 16, and the leading byte
// offset / 16 from bit 16; the high one: stride byte offset 1024 / 16, version 1, 128-byte
// swizzle.  K-major operands (Q, K: 128-byte rows, 8-row groups 1024 bytes apart) leave the
// leading byte offset unused; V, N-major (64 dims contiguous per key, 8-key groups 1024 bytes
// apart), finds its second 64 dims there, kHalfTile further.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescK = 1u << 16, kDescV = (kHalfTile >> 4) << 16;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t base) { return base | ((saddr & 0x3FFFFu) >> 4); }

// D += A B, A and B in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(kDescHi)
      : "memory");
}
// D += A B with A (bf16 pairs, one 32-bit column per two K) in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(kDescHi)
      : "memory");
}

// One thread of the (whole, converged) warp, always the same.  Code under it is known to run
// on one lane, with the warp's uniform values in uniform registers: MMAs issued under a test
// of the lane number instead cost 120 cycles each for a pipe that takes one in 64.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

#define R4(b, i) "=r"(b[i]), "=r"(b[i + 1]), "=r"(b[i + 2]), "=r"(b[i + 3])
#define R16(b, i) R4(b, i), R4(b, i + 4), R4(b, i + 8), R4(b, i + 12)
// 32 columns of this warp's 32 lanes, asynchronous until tmem_wait_ld
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : R16(r, 0), R16(r, 16)
      : "r"(addr));
}
#undef R4
#undef R16
// 16 columns
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void fma2(float &x, float &y, float s, float t) {   // (x, y) * s + t
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %3};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(s), "f"(t));
}
__device__ __forceinline__ void add2(float &x, float &y, float s, float t) {   // (x, y) + (s, t)
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(s), "f"(t));
}

// A range's part of one item: key tiles from the place on.
__device__ __forceinline__ int seg_tiles(const Place &p, int left) { return min(p.s.n - p.j, left); }
__device__ __forceinline__ int group_rows(const Args &a, const Place &p) { return p.u < 0 ? a.prows : a.rows; }
// (shared form) whether the row tile has rows in its second half
__device__ __forceinline__ bool two_halves(const Args &a, const Place &p) {
  return group_rows(a, p) - p.rt * 256 > 128;
}

// Every lane waits; the warp carries on only if all of them saw the phase complete.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = wait_bar(bar, parity, abort_flag, status);
  return __all_sync(0xffffffffu, ok);
}

// The same for three phases, asked for together.  (A wait that need not wait costs 170 cycles,
// most of them the answer's way; four in a row, and the checks between them, made the loop
// of the MMA warps 1830 cycles a tile, longer than the products.)
__device__ __forceinline__ bool warp_wait3(uint32_t bar0, uint32_t par0, uint32_t bar1, uint32_t par1, uint32_t bar2,
                                           uint32_t par2, volatile int *abort_flag, int *status) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6;\n\t"
      "and.pred p, p, q;\n\tand.pred p, p, r;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(bar0), "r"(par0), "r"(bar1), "r"(par1), "r"(bar2), "r"(par2)
      : "memory");
  if (__all_sync(0xffffffffu, r != 0)) return true;
  const bool ok = wait_bar(bar0, par0, abort_flag, status) && wait_bar(bar1, par1, abort_flag, status) &&
                  wait_bar(bar2, par2, abort_flag, status);
  return __all_sync(0xffffffffu, ok);
}

template <bool kTwo>   // the streams form
__global__ void __launch_bounds__(kThreads, 1) ragged_tc_kernel(const __grid_constant__ TcParams prm) {
  constexpr int kRW = kTwo ? kStreamRows : kSharedRows;
  const Args &a = prm.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t qs = (raw + 1023u) & ~1023u;
  const uint32_t ring = qs + kQBytes;
  uint8_t *sq = smem_raw + (qs - raw);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sq + kQBytes + kStages * kTileBytes);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages;
  // per half and buffer of Q: there, no longer needed (streams); per half: S there, S read; per
  // half and buffer of P: P there, added to O
  const uint32_t qfull0 = empty0 + 8 * kStages, qfree0 = qfull0 + 32, sfull0 = qfree0 + 32, sfree0 = sfull0 + 16;
  const uint32_t pfull0 = sfree0 + 16, pdone0 = pfull0 + 32, drain_bar = pdone0 + 32;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 2 * kStages + 22);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    prefetch_map(&prm.k);
    prefetch_map(&prm.v);
    if (a.PRT > 0) {
      prefetch_map(&prm.kp);
      prefetch_map(&prm.vp);
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, kTwo ? 1 : 2);   // the halves that use it
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(sfull0 + 8 * h, 1);
      mbar_init(sfree0 + 8 * h, 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(qfull0 + 16 * h + 8 * b, kTwo ? 1 : 4);
        mbar_init(qfree0 + 16 * h + 8 * b, 4);
        mbar_init(pfull0 + 16 * h + 8 * b, 4);
        mbar_init(pdone0 + 16 * h + 8 * b, 1);
      }
    }
    mbar_init(drain_bar, 1);
    mbar_init(drain_bar + 8, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
  wait_first(a);
  pdl_release();

  // the half that this warp serves (shared form, warp 8: both)
  const int h = warp < 8 ? warp >> 2 : (warp == 8 || warp == 9 ? 0 : 1);
  const int cta = blockIdx.x / a.nkv, g = blockIdx.x - cta * a.nkv;
  const int range = kTwo ? 2 * cta + h : cta;
  int x0 = 0, left = 0;
  Place p = {};
  find_range<kRW, kKT>(a, range, p, x0, left);
  // this half's stages of the ring
  constexpr int S = kTwo ? kStages / 2 : kStages;
  const int stage0 = kTwo ? S * h : 0;

  if (warp == 8 || warp == 11) {
    // ---------------------------------------------------------------- key and value tiles
    if (lane == 0 && (kTwo || warp == 8)) {
      const uint64_t pol = kTwo ? policy_evict_first() : policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0, items = 0;
      bool ok = true, fresh = true;
      for (; left > 0 && ok; --left) {
        if (kTwo && fresh) {   // the item's rows of q: all heads of the group, all queries
          if (items >= 2) ok = wait_bar(qfree0 + 16 * h + 8 * (items & 1), ((items >> 1) - 1) & 1, abort_flag, a.status);
          if (!ok) break;
          const uint32_t fb = qfull0 + 16 * h + 8 * (items & 1), dst = qs + (h * 2 + (items & 1)) * 64 * 128;
          const CUtensorMap *mq = p.u < 0 ? &prm.qp : &prm.q;
          const int i0 = p.u < 0 ? 0 : p.u * a.nr;
          mbar_expect_tx(fb, group_rows(a, p) * kHD * 2);
          tma_load_3d(dst, mq, 0, g * a.grp, i0, fb, policy_evict_last());
          tma_load_3d(dst + kQHalf, mq, 64, g * a.grp, i0, fb, policy_evict_last());
          ++items;
        }
        fresh = p.j + 1 == p.s.n;
        const int t0 = tile_key<kKT>(p);
        const CUtensorMap *mk = p.u < 0 ? &prm.kp : &prm.k, *mv = p.u < 0 ? &prm.vp : &prm.v;
        const int b = p.u < 0 ? 0 : p.u;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          if (ok && !wait_bar(empty0 + 8 * (stage0 + stage), phase ^ 1u, abort_flag, a.status)) ok = false;
          if (!ok) break;
          const uint32_t fb = full0 + 8 * (stage0 + stage), dst = ring + (stage0 + stage) * kTileBytes;
          mbar_expect_tx(fb, kTileBytes);
          tma_load_4d(dst, which ? mv : mk, 0, g, t0, b, fb, pol);
          tma_load_4d(dst + kHalfTile, which ? mv : mk, 64, g, t0, b, fb, pol);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (left > 1) next_unit<kRW, kKT>(a, p);
      }
      if (!ok) {   // let the copies already issued land before the CTA exits
        for (int j = items > 2 ? items - 2 : 0; kTwo && j < items; ++j) {
          const long long c0 = clock64();
          while (!mbar_try_wait(qfull0 + 16 * h + 8 * (j & 1), static_cast<uint32_t>((j >> 1) & 1)) &&
                 clock64() - c0 < kWaitCycles) {
          }
        }
        for (int j = issued > S ? issued - S : 0; j < issued; ++j) {
          const long long c0 = clock64();
          while (!mbar_try_wait(full0 + 8 * (stage0 + j % S), static_cast<uint32_t>((j / S) & 1)) && clock64() - c0 < kWaitCycles) {
          }
        }
      }
    }
  } else if (warp > 8) {
    // ---------------------------------------------------------------- one half's MMAs
    const uint32_t ts = tmem + h * 64, tp = tmem + 128 + h * 64, to = tmem + 256 + h * 128;
    int stage = 0;          // of the next tile to be used
    uint32_t phase = 0, sph = 0;
    int count = 0, items = 0;   // tiles and items of this half so far
    bool ok = true;
    auto next_stage = [&](int &s, uint32_t &ph) {   // the next tile of the ring
      s = stage0 + stage;
      ph = phase;
      if (++stage == S) {
        stage = 0;
        phase ^= 1u;
      }
    };
    uint32_t q_lo = desc_lo(qs + h * 128 * 128, kDescK);
    auto qk = [&](int s) {   // S of the tile in stage s
      tc_fence_after();
      if (elect_one()) {
        const uint32_t k_lo = desc_lo(ring + s * kTileBytes, kDescK);
#pragma unroll
        for (int kk = 0; kk < kHD / 16; ++kk)   // 32 bytes of a row, then the second 64 dims
          mma_ss(ts, q_lo + (kk >> 2) * (kQHalf >> 4) + (kk & 3) * 2, k_lo + (kk >> 2) * (kHalfTile >> 4) + (kk & 3) * 2,
                 kIdesc, kk > 0);
        tc_commit(sfull0 + 8 * h);
        tc_commit(empty0 + 8 * s);
      }
      __syncwarp();
    };
    while (left > 0 && ok) {
      const int n = seg_tiles(p, left);
      int ks, vs;
      uint32_t kph, vph;
      if (!kTwo && h == 1 && !two_halves(a, p)) {   // no rows here: the tiles pass by
        for (int t = 0; t < 2 * n && ok; ++t) {
          next_stage(ks, kph);
          ok = warp_wait(full0 + 8 * ks, kph, abort_flag, a.status);
          if (ok && lane == 0) mbar_arrive(empty0 + 8 * ks);
        }
      } else {
        next_stage(ks, kph);
        ok = warp_wait(full0 + 8 * ks, kph, abort_flag, a.status);
        if (ok && count > 0) {   // S of the item before has been read
          ok = warp_wait(sfree0 + 8 * h, sph, abort_flag, a.status);
          sph ^= 1u;
        }
        if (!ok) break;
        const int qb = kTwo ? items & 1 : 0;
        ok = warp_wait(qfull0 + 16 * h + 8 * qb, (kTwo ? items >> 1 : items) & 1, abort_flag, a.status);
        if (!ok) break;
        if (kTwo) q_lo = desc_lo(qs + (h * 2 + qb) * 64 * 128, kDescK);
        ++items;
        qk(ks);
        const int sinks = p.u < 0 ? 0 : a.sinks;
        for (int t = 0; t < n && ok; ++t) {
          const int b = count & 1;
          const uint32_t pph = (count >> 1) & 1;
          ++count;
          next_stage(vs, vph);
          if (t + 1 < n) {   // Q K^T of the next tile: its keys there, S read
            next_stage(ks, kph);
            ok = warp_wait3(full0 + 8 * ks, kph, sfree0 + 8 * h, sph, full0 + 8 * vs, vph, abort_flag, a.status);
            sph ^= 1u;
            if (!ok) break;
            qk(ks);
          } else {
            ok = warp_wait(full0 + 8 * vs, vph, abort_flag, a.status);
            if (!ok) break;
          }
          Place q = p;
          q.j = p.j + t;
          const int t0 = tile_key<kKT>(q);
          uint32_t steps = 0xfu;   // steps of 16 keys of which some row sees one
          if (t0 + kKT > p.s.hi || (t0 < p.s.lo && t0 + kKT > sinks)) {
            auto seen = [&](int key) { return key < p.s.hi && (key >= p.s.lo || key < sinks); };
            const int k2 = t0 + 2 * lane;   // this lane's two keys
            const bool s0 = seen(k2), s1 = seen(k2 + 1);
            const uint32_t any = __ballot_sync(0xffffffffu, s0 || s1);
            const uint32_t all = __ballot_sync(0xffffffffu, s0 && s1);
            steps = 0;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t some = (any >> (8 * kk)) & 255u;
              if (some) steps |= 1u << kk;
              if (some && ((all >> (8 * kk)) & 255u) != 255u) {
                uint4 *vt = reinterpret_cast<uint4 *>(sq + kQBytes + vs * kTileBytes);
#pragma unroll
                for (int i = 0; i < 8; ++i) {   // two rows at a time, 16 chunks each
                  const int r = 16 * kk + 2 * i + (lane >> 4);
                  if (!seen(t0 + r))
                    vt[((lane >> 3) & 1) * (kHalfTile / 16) + r * 8 + (lane & 7)] = make_uint4(0u, 0u, 0u, 0u);
                }
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          ok = warp_wait(pfull0 + 16 * h + 8 * b, pph, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t v_lo = desc_lo(ring + vs * kTileBytes, kDescV), pt = kTwo ? tp : tp + b * 32;
            if (steps == 0xfu) {
#pragma unroll
              for (int part = 0; part < (kTwo ? 2 : 1); ++part)
#pragma unroll
                for (int kk = 0; kk < kKT / 16; ++kk)
                  mma_ts(to, pt + part * 32 + kk * 8, v_lo + kk * (2048 >> 4), kIdescPV, t > 0 || part > 0 || kk > 0);
            } else {
              bool acc = t > 0;
#pragma unroll 1
              for (int kk = 0; kk < kKT / 16; ++kk)
                if ((steps >> kk) & 1u) {
                  mma_ts(to, pt + kk * 8, v_lo + kk * (2048 >> 4), kIdescPV, acc);
                  acc = true;
                  if (kTwo) mma_ts(to, pt + 32 + kk * 8, v_lo + kk * (2048 >> 4), kIdescPV, true);
                }
            }
            tc_commit(pdone0 + 16 * h + 8 * b);
            tc_commit(empty0 + 8 * vs);
          }
          __syncwarp();
        }
      }
      left -= n;
      if (left > 0) next_item<kRW, kKT>(a, p);
    }
    __syncwarp();
    if (elect_one()) {   // every MMA of this half has completed once this arrives
      tc_commit(drain_bar + 8 * h);
      const long long c0 = clock64();
      while (!mbar_try_wait(drain_bar + 8 * h, 0) && clock64() - c0 < kWaitCycles) {
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax of one half
    const int quarter = warp & 3;
    const int row_in = (kTwo ? 0 : h * 128) + quarter * 32 + lane;   // row of the tile
    const bool has_q = row_in - lane < kRW;                           // this warp has rows of the tile
    // this warp's 32 rows of Q: 4 KB in each of the two dims' halves
    uint8_t *sw = sq + (h * 128 + quarter * 32) * 128;
    int items = 0;            // items of this half so far
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_addr + h * 64, tp = tmem + lane_addr + 128 + h * 64;
    const uint32_t to = tmem + lane_addr + 256 + h * 128;
    int count = 0;            // tiles of this half so far
    bool ok = true, first_item = true;
    // the segment whose output is still in tensor memory
    bool pending = false, pend_whole = false, pend_valid = false;
    int64_t pend_dst = 0;     // its row of out (whole) or of the pieces
    int pend_src = 0;         // whole rows over a prefix: 0 prefix, 1 own keys
    float m = -INFINITY, l = 0.0f;

    auto added = [&](int i) {   // waits until tile i's P V has been added to O
      return warp_wait(pdone0 + 16 * h + 8 * (i & 1), (i >> 1) & 1, abort_flag, a.status);
    };
    auto finish = [&]() {     // O of the pending segment to memory
      ok = added(count - 1);
      tc_fence_after();
      if (!ok || !has_q) return;
      const bool to_out = pend_whole && a.P == 0;
      float *po = nullptr;
      float2 *pm = nullptr;
      if (!pend_whole) {
        po = a.part_o;
        pm = a.part_ml + pend_dst;
      } else if (a.P > 0) {
        const int64_t src = pend_src ? static_cast<int64_t>(a.B) * a.nr * a.nq : 0;
        po = a.row_o + src * kHD;
        pm = a.row_ml + src + pend_dst;
      }
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      // 32 columns at a time through the warp's own 4 KB of Q (its products are done), so
      // that eight lanes store 128 bytes of a row (16 bytes of 32 rows per store took 7 to 12
      // thousand cycles an item)
      const int64_t off = pend_valid ? pend_dst * kHD : -1;
#pragma unroll 1
      for (int c = 0; c < kHD; c += 32) {
        uint32_t r[32];
        tmem_ld32(to + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)   // 16-byte chunk i of row `lane` at chunk i ^ (lane & 7)
          *reinterpret_cast<uint4 *>(sw + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3);
          const uint4 x = *reinterpret_cast<const uint4 *>(sw + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
          const int64_t o = __shfl_sync(0xffffffffu, off, rr);
          const float f = __shfl_sync(0xffffffffu, inv, rr);
          if (o < 0) continue;
          if (to_out)
            *reinterpret_cast<uint2 *>(a.out + o + c + 4 * (lane & 7)) =
                make_uint2(pack_bf16(__uint_as_float(x.x) * f, __uint_as_float(x.y) * f),
                           pack_bf16(__uint_as_float(x.z) * f, __uint_as_float(x.w) * f));
          else
            *reinterpret_cast<uint4 *>(po + o + c + 4 * (lane & 7)) = x;
        }
        __syncwarp();
      }
      if (pend_valid && !to_out) *pm = make_float2(m, l);
      if (pend_valid && to_out && a.row_ml) a.row_ml[pend_dst] = make_float2(m, inv);   // scored
    };

    while (left > 0 && ok) {
      const int n = seg_tiles(p, left);
      const int grows = group_rows(a, p);
      const bool mine = kTwo || h == 0 || two_halves(a, p);
      if (mine) {
        const int r = p.rt * kRW + row_in;
        const bool valid = row_in < kRW && r < grows;
        const int64_t qrow = q_row(a, p.u, g, valid ? r : 0);
        if (kTwo) {
          sw = sq + ((h * 2 + (items & 1)) * 64 + quarter * 32) * 128;
        } else {
          // the item's Q, half of it on its way while the one before is finished (all of it
          // would not fit in the registers); two rows per load, 16 lanes each (a row past the
          // last one: zeros)
          const int64_t off = valid ? qrow * kHD : -1;
          uint4 x[8];
          auto load_q = [&](int i0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t o = __shfl_sync(0xffffffffu, off, 2 * (i0 + i) + (lane >> 4));
              x[i] = o >= 0 ? *reinterpret_cast<const uint4 *>(a.q + o + 8 * (lane & 15)) : make_uint4(0u, 0u, 0u, 0u);
            }
          };
          auto store_q = [&](int i0) {
            const int c = lane & 15;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = 2 * (i0 + i) + (lane >> 4);
              *reinterpret_cast<uint4 *>(sw + (c >> 3) * kQHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = x[i];
            }
          };
          load_q(0);
          if (pending) finish();
          if (!ok) break;
          store_q(0);   // (this half's Q may be overwritten: its last S has arrived)
          load_q(8);
          store_q(8);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(qfull0 + 16 * h);
        }
        m = -INFINITY;
        l = 0.0f;
        int lo = 0, hi = 0x7fffffff;
        if (valid) row_bounds(a, p.u, p.len, r, lo, hi);
        const int sinks = p.u < 0 ? 0 : a.sinks;
        const bool active = __any_sync(0xffffffffu, valid);
        Place q = p;
        for (int t = 0; t < n; ++t, ++count) {
          q.j = p.j + t;
          const int t0 = tile_key<kKT>(q);
          const bool open = __all_sync(0xffffffffu, t0 >= lo && t0 + kKT <= hi);
          ok = warp_wait(sfull0 + 8 * h, count & 1, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          uint32_t sr[kKT];   // scores, then pairs of weights from the front
          if (active) {
            tmem_ld32(ts, sr);
            tmem_ld32(ts + 32, sr + 32);
            tmem_wait_ld();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sfree0 + 8 * h);
          if (active) {
            if (!open) {
              // keys a row does not see count as -inf: bit c of a mask says whether key k + c counts
              auto below = [](int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); };
#pragma unroll
              for (int c0 = 0; c0 < kKT; c0 += 32) {
                const int k = t0 + c0;
                const uint32_t seen = below(hi - k) & (~below(lo - k) | below(sinks - k));
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!((seen >> c) & 1u)) sr[c0 + c] = 0xff800000u;
              }
            }
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(sr[i]);
#pragma unroll
            for (int c = 4; c < kKT; c += 4)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = fmaxf(x[i], __uint_as_float(sr[c + i]));
            const float top = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * a.scale_log2);
            if (t == 0) {
              m = top;
            } else if (__any_sync(0xffffffffu, valid && top > m + kRescale)) {
              // (a row that had seen no key yet: m + 8 is -inf, its O and sum are zeros)
              ok = added(count - 1);
              if (!ok) break;
              tc_fence_after();
              const float f = top == -INFINITY ? 1.0f : ex2(m - top);
              l *= f;
              m = top;
#pragma unroll 1
              for (int c = 0; c < kHD; c += 16) {
                uint32_t r[16];
                tmem_ld16(to + c, r);
#pragma unroll
                for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                tmem_st16(to + c, r);
              }
            }
            const float nm = m == -INFINITY ? 0.0f : -m;
            float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
            uint32_t low[kTwo ? kKT / 2 : 1];
#pragma unroll
            for (int c = 0; c < kKT; c += 4) {
              float e[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] = __uint_as_float(sr[c + i]);
              fma2(e[0], e[1], a.scale_log2, nm);
              fma2(e[2], e[3], a.scale_log2, nm);
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] = ex2(e[i]);
              add2(s0, s1, e[0], e[1]);
              add2(s2, s3, e[2], e[3]);
              sr[c / 2] = pack_bf16(e[0], e[1]);
              sr[c / 2 + 1] = pack_bf16(e[2], e[3]);
              if (kTwo) {
                low[c / 2] = pack_bf16(e[0] - bf16_lo(sr[c / 2]), e[1] - bf16_hi(sr[c / 2]));
                low[c / 2 + 1] = pack_bf16(e[2] - bf16_lo(sr[c / 2 + 1]), e[3] - bf16_hi(sr[c / 2 + 1]));
              }
            }
            l += (s0 + s1) + (s2 + s3);
            if (kTwo) {
              // hi and lo fill both buffers: the tile before has to be added to O first (an
              // item's first tile: the item before was finished)
              if (t > 0) ok = added(count - 1);
              if (!ok) break;
              tc_fence_after();
              tmem_st16(tp, sr);
              tmem_st16(tp + 16, sr + 16);
              tmem_st16(tp + 32, low);
              tmem_st16(tp + 48, low + 16);
            } else {
              // (this buffer's last tile, the one before last, has been added to O: its P V was
              // issued before this tile's Q K^T, whose commit covers it)
              tmem_st16(tp + (count & 1) * 32, sr);
              tmem_st16(tp + (count & 1) * 32 + 16, sr + 16);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull0 + 16 * h + 8 * (count & 1));
        }
        if (!ok) break;
        pending = true;
        pend_whole = n == p.s.n;
        pend_valid = valid;
        pend_src = p.u < 0 ? 0 : 1;
        pend_dst = pend_whole ? qrow
                              : (static_cast<int64_t>(range * a.nkv + g) * 2 + (first_item ? 0 : 1)) * kRW + row_in;
        if (kTwo) {
          finish();
          if (!ok) break;
          // (the staging is read before this buffer's next Q is written by the async proxy)
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(qfree0 + 16 * h + 8 * (items & 1));
          ++items;
        }
      }
      first_item = false;
      left -= n;
      if (left > 0) next_item<kRW, kKT>(a, p);
    }
    if (!kTwo && pending && ok) finish();
    tc_fence_before();
  }

  __syncwarp();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
  wait_last(a);
}

// [rows, nq, 128] bf16 in boxes of 64 dims of `heads` heads of n rows
bool rows_map(CUtensorMap *map, const void *ptr, int rows, int nq, int heads, int n) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {kHD, static_cast<cuuint64_t>(nq), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {kHD * 2, static_cast<cuuint64_t>(nq) * kHD * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(n)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

dspark_status_t tc_launch(const Args &a, Form form, cudaStream_t stream) {
  TcParams prm;
  prm.a = a;
  if (!cache_map(&prm.k, a.k_cache, a.B, a.cache_len, a.nkv, kKT) ||
      !cache_map(&prm.v, a.v_cache, a.B, a.cache_len, a.nkv, kKT))
    return DSPARK_ERR_UNSUPPORTED_SHAPE;
  prm.kp = prm.k;
  prm.vp = prm.v;
  if (a.PRT > 0 && (!cache_map(&prm.kp, a.k_prefix, 1, a.P, a.nkv, kKT) || !cache_map(&prm.vp, a.v_prefix, 1, a.P, a.nkv, kKT)))
    return DSPARK_ERR_UNSUPPORTED_SHAPE;
  const bool streams = form == kStreams;
  if (streams) {
    if (!rows_map(&prm.q, a.q, a.B * a.nr, a.nq, a.grp, a.nr)) return DSPARK_ERR_CUDA;
    prm.qp = prm.q;
    if (a.PRT > 0 && !rows_map(&prm.qp, a.q, a.B * a.nr, a.nq, a.grp, a.B * a.nr)) return DSPARK_ERR_CUDA;
  }
  auto kern = streams ? ragged_tc_kernel<true> : ragged_tc_kernel<false>;
  static std::atomic<bool> done[2][64];
  if (!allow_smem(kern, kSmem, done[streams])) return DSPARK_ERR_CUDA;
  const int ctas = (streams ? (a.groups + 1) / 2 : a.groups) * a.nkv;
  if (launch_kernel(!a.ordinary, kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), kSmem, stream, prm) !=
      cudaSuccess)
    return DSPARK_ERR_CUDA;
  count_launches(1);
  return DSPARK_OK;
}

}  // namespace ragged
}  // namespace dspark
