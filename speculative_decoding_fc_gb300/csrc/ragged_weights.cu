// The scored attention's second pass over the keys for groups of 17 to 64 query rows: with
// every row's maximum M and 1 / sum known,
//   scores_out[b, g, t] = decay * scores_in[b, g, t] + sum_r e^(s[r, t] - M_r) / L_r
// over the group's rows r that see key t.  The scores are formed again, transposed: S^T =
// K Q^T with a tile of 128 keys as the MMA's M and the rows (padded to 16) as its N, so that
// a key is one thread's and its sum needs no exchange between threads.  It reads the keys
// once more (256 bytes a key; from L2 while the batch's keys fit there); keeping the first
// pass's scores instead would write and read 8 bytes a key for every row (320 at 40 rows),
// in a workspace of that size.  Bound by the keys' reading when there are many; one request of
// 2057 keys and 8 kv heads takes 10.5 us, most of it the start (plan, maps, Q, one tile each).
// One CTA per SM and range: warps 0-3 sum (one thread per key), warp 4 loads (TMA, ring of five 32 KB tiles), warp 5 issues the MMAs into
// two accumulators.  Waits are bounded as in gemm_tcgen05.cu.
#include "common.cuh"
#include "internal.h"
#include "ragged.cuh"
#include "ragged_host.h"
#include "tcgen05.cuh"

namespace dspark {
namespace ragged {

using namespace tc;

struct WeightParams {
  Args a;
  CUtensorMap k;
};

namespace {

constexpr int kKT = kWeightKeys, kRW = kStreamRows;
constexpr int kThreads = 192;
constexpr int kStages = 5;
constexpr uint32_t kHalfTile = kKT * 128;
constexpr uint32_t kTileBytes = 2 * kHalfTile;
constexpr uint32_t kQHalf = kMaxScoredRows * 128;       // [64 rows][64 dims]
constexpr uint32_t kQBytes = 2 * kQHalf;
constexpr uint32_t kStatBytes = kMaxScoredRows * 16;    // per row: M, 1 / L, first key it does not see
constexpr uint32_t kSmem = 1024 + 2 * kQBytes + kStages * kTileBytes + 4 * kStatBytes + 256;

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = wait_bar(bar, parity, abort_flag, status);
  return __all_sync(0xffffffffu, ok);
}

__global__ void __launch_bounds__(kThreads, 1) ragged_weights_kernel(const __grid_constant__ WeightParams prm) {
  const Args &a = prm.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t qs = (raw + 1023u) & ~1023u;           // two Q buffers, then the ring
  const uint32_t ring = qs + 2 * kQBytes;
  uint8_t *sq = smem_raw + (qs - raw);
  float4 *stats = reinterpret_cast<float4 *>(sq + 2 * kQBytes + kStages * kTileBytes);
  uint64_t *bars = reinterpret_cast<uint64_t *>(stats + 4 * kMaxScoredRows);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kStages;
  const uint32_t qfull0 = empty0 + 8 * kStages, tfull0 = qfull0 + 16, tempty0 = tfull0 + 16, drain_bar = tempty0 + 16;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 2 * kStages + 7);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(qfull0 + 8 * i, 4);
      mbar_init(tfull0 + 8 * i, 1);
      mbar_init(tempty0 + 8 * i, 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(128u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  pdl_release();

  const int cta = blockIdx.x / a.nkv, g = blockIdx.x - cta * a.nkv;
  int x0 = 0, left = 0;
  Place p = {};
  find_range<kRW, kKT>(a, cta, p, x0, left);
  const int N = (a.rows + 15) / 16 * 16;

  if (warp == 4) {
    // ---------------------------------------------------------------- keys
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (; left > 0; --left) {
        ok = wait_bar(empty0 + 8 * stage, phase ^ 1u, abort_flag, a.status);
        if (!ok) break;
        const uint32_t fb = full0 + 8 * stage, dst = ring + stage * kTileBytes;
        const int t0 = tile_key<kKT>(p);
        mbar_expect_tx(fb, kTileBytes);
        tma_load_4d(dst, &prm.k, 0, g, t0, p.u, fb, pol);
        tma_load_4d(dst + kHalfTile, &prm.k, 64, g, t0, p.u, fb, pol);
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (left > 1) next_unit<kRW, kKT>(a, p);
      }
      if (!ok)   // let the copies already issued land before the CTA exits
        for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j) {
          const long long c0 = clock64();
          while (!mbar_try_wait(full0 + 8 * (j % kStages), static_cast<uint32_t>((j / kStages) & 1)) &&
                 clock64() - c0 < kWaitCycles) {
          }
        }
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMAs
    if (lane == 0) {
      // D fp32, A and B bf16 K-major, M = 128
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
      int stage = 0, acc = 0, item = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      while (left > 0 && ok) {
        const int n = min(p.s.n - p.j, left);
        ok = wait_bar(qfull0 + 8 * (item & 1), (item >> 1) & 1, abort_flag, a.status);
        const uint32_t q = qs + (item & 1) * kQBytes;
        for (int t = 0; t < n && ok; ++t) {
          ok = wait_bar(tempty0 + 8 * acc, acc_phase ^ 1u, abort_flag, a.status) &&
               wait_bar(full0 + 8 * stage, phase, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k = ring + stage * kTileBytes;
#pragma unroll
          for (int kk = 0; kk < kHD / 16; ++kk) {
            const uint32_t off = (kk & 3) * 32;
            tc_mma_bf16(tmem + acc * 64, sdesc_k_sw128(k + (kk >> 2) * kHalfTile + off),
                        sdesc_k_sw128(q + (kk >> 2) * kQHalf + off), idesc, kk > 0 ? 1u : 0u);
          }
          tc_commit(empty0 + 8 * stage);
          tc_commit(tfull0 + 8 * acc);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
        left -= n;
        ++item;
        if (left > 0) next_item<kRW, kKT>(a, p);
      }
      tc_commit(drain_bar);
      const long long c0 = clock64();
      while (!mbar_try_wait(drain_bar, 0) && clock64() - c0 < kWaitCycles) {
      }
    }
  } else {
    // ---------------------------------------------------------------- sums, one thread per key
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // rows 16 w .. 16 w + 15 of item i: q (two buffers, read by the MMAs only) and the rows'
    // statistics (four: a warp can be two tiles, and so two items, behind the others)
    auto load_rows = [&](const Place &at, int i_item) {
      const int r0 = warp * 16, buf = i_item & 1;
      const int c = lane & 15;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + 2 * i + (lane >> 4);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < a.rows) x = *reinterpret_cast<const uint4 *>(a.q + q_row(a, at.u, g, r) * kHD + 8 * c);
        *reinterpret_cast<uint4 *>(sq + buf * kQBytes + (c >> 3) * kQHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
      }
      if (lane < 16) {
        const int r = r0 + lane;
        float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < a.rows) {
          const float2 ml = __ldcg(a.row_ml + q_row(a, at.u, g, r));
          int lo, hi;
          row_bounds(a, at.u, at.len, r, lo, hi);
          if (ml.x != -INFINITY) st = make_float4(ml.x, ml.y, __int_as_float(hi), 0.0f);
        }
        stats[(i_item & 3) * kMaxScoredRows + r] = st;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull0 + 8 * buf);
    };
    int acc = 0, item = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    if (left > 0) load_rows(p, 0);
    while (left > 0 && ok) {
      const int n = min(p.s.n - p.j, left);
      Place next = p;
      if (left > n) {
        // the next item's rows: their buffer's MMAs (the item before this one) are done,
        // all of its sums have been taken
        next_item<kRW, kKT>(a, next);
        load_rows(next, item + 1);
      }
      // the four warps' statistics of this item
      ok = warp_wait(qfull0 + 8 * (item & 1), (item >> 1) & 1, abort_flag, a.status);
      if (!ok) break;
      const float4 *st = stats + (item & 3) * kMaxScoredRows;
      for (int t = 0; t < n; ++t, ++p.j) {
        ok = warp_wait(tfull0 + 8 * acc, acc_phase, abort_flag, a.status);
        if (!ok) break;
        tc_fence_after();
        const int key = tile_key<kKT>(p) + warp * 32 + lane;
        float w = 0.0f;
        for (int c = 0; c < N; c += 16) {
          uint32_t r[16];
          tmem_ld16(lane_addr + acc * 64 + c, r);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float4 v = st[c + i];
            const float e = ex2(__fmaf_rn(__uint_as_float(r[i]), a.scale_log2, -v.x)) * v.y;
            w += key < __float_as_int(v.z) ? e : 0.0f;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
        if (key < p.len) {
          const int64_t at = (static_cast<int64_t>(p.u) * a.nkv + g) * a.cache_len + key;
          if (a.scores_in) w = __fmaf_rn(a.decay, a.scores_in[at], w);
          a.scores_out[at] = w;
        }
      }
      left -= n;
      ++item;
      p = next;
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(128u) : "memory");
  }
}

}  // namespace

dspark_status_t weights_launch(const Args &a, cudaStream_t stream) {
  WeightParams prm;
  prm.a = a;
  if (!cache_map(&prm.k, a.k_cache, a.B, a.cache_len, a.nkv, kKT)) return DSPARK_ERR_UNSUPPORTED_SHAPE;
  static std::atomic<bool> done[64];
  if (!allow_smem(ragged_weights_kernel, kSmem, done)) return DSPARK_ERR_CUDA;
  if (launch_pdl(ragged_weights_kernel, dim3(static_cast<unsigned>(a.groups * a.nkv)), dim3(kThreads), kSmem,
                 stream, prm) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  count_launches(1);
  return DSPARK_OK;
}

}  // namespace ragged
}  // namespace dspark
