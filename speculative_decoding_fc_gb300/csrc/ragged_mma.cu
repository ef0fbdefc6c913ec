// Attention over ragged key/value caches, at most 16 query rows per kv head (single tokens,
// short blocks): the decode kernel, which reads the keys and values once at the memory's
// rate, and the kernels around it: the plan, the joining of split items and the column sums
// of the scored form.  Schedule and masks: ragged.cuh.
#include "common.cuh"
#include "internal.h"
#include "ragged.cuh"
#include "ragged_host.h"
#include "tcgen05.cuh"

namespace dspark {
namespace ragged {

using namespace tc;

struct MmaParams {
  Args a;
  CUtensorMap k, v, kp, vp;
};

namespace {

static_assert(kMmaKeys == kTcKeys, "the joins take one key tile for both kernels");
constexpr int kKT = kMmaKeys;                           // keys per tile
constexpr int kRW = kMmaRows;
constexpr int kThreads = 128;                           // 4 warps
constexpr int kStages = 3;
constexpr uint32_t kHalfTile = kKT * 128;               // [64 keys][64 dims] bf16
constexpr uint32_t kTileBytes = 2 * kHalfTile;          // one of K, V
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + 64;
constexpr int kMergeFloats = kRW * kHD + 2 * kRW;       // one warp's rows: o, m, l

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the bf16 parts hi = bf16(x), lo = bf16(x - hi) of two weights
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(x0, x1);
  lo = pack_bf16(x0 - bf16_lo(hi), x1 - bf16_hi(hi));
}

// CTA (range, kv head).  Warp w takes keys 16 w .. 16 w + 15 of each tile for all 16 rows,
// with its own running maximum, sum and output: the warps' results meet only at the item's
// end.  16 rows are one warp-level MMA's height; the tcgen05 MMA's is 128, and with 5 rows
// of a group there would be nothing but padding in it, which costs its softmax's registers
// and latency.  Scores: bf16 q and k, fp32 sums, log2 units (scaled by log2(e) / sqrt(128)
// after the sum).  The weights enter P.V as bf16 parts hi + lo (2^-16 relative; the kernel
// waits for memory, the second product costs nothing), the value rows exact.
// One thread issues a tile's loads (TMA, four boxes of 64 keys x 64 dims in 128-byte
// swizzle, which ldmatrix reads without conflicts): copies issued by every thread
// (cp.async) took 1000 to 1500 cycles of a tile's 2900.  Keys outside the item's span count
// as -inf; their value rows are zeroed in shared memory, whatever they hold.
// Bound by the memory: 64 single tokens over 230 MB of keys and values 43 us cold (5.4 TB/s),
// 32 over 379 MB with the row scores stored 62 us (6.1 TB/s); what is missing to the copy's
// rate is the first tiles' wait and the ends of items (230 registers, two CTAs of four warps).
template <bool kScored>
__global__ void __launch_bounds__(kThreads, 2) ragged_mma_kernel(const __grid_constant__ MmaParams prm) {
  const Args &a = prm.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t *sring = smem_raw + (ring - raw);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sring + kStages * kStageBytes);
  const uint32_t full0 = smem_u32(bars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kStages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full0 + 8 * s, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    prefetch_map(&prm.k);
    prefetch_map(&prm.v);
  }
  __syncthreads();
  wait_first(a);
  pdl_release();

  const int range = blockIdx.x / a.nkv, g = blockIdx.x - range * a.nkv;
  Place cp = {};
  int x0 = 0, units;
  find_range<kRW, kKT>(a, range, cp, x0, units);
  if (units == 0) {
    wait_last(a);
    return;
  }
  Place ld = cp;

  const uint64_t pol = policy_evict_first();
  auto load_tile = [&](const Place &p, int stage) {   // by one thread
    const int t0 = tile_key<kKT>(p), b = p.u < 0 ? 0 : p.u;
    const CUtensorMap *mk = p.u < 0 ? &prm.kp : &prm.k, *mv = p.u < 0 ? &prm.vp : &prm.v;
    const uint32_t dst = ring + stage * kStageBytes, bar = full0 + 8 * stage;
    mbar_expect_tx(bar, kStageBytes);
    tma_load_4d(dst, mk, 0, g, t0, b, bar, pol);
    tma_load_4d(dst + kHalfTile, mk, 64, g, t0, b, bar, pol);
    tma_load_4d(dst + kTileBytes, mv, 0, g, t0, b, bar, pol);
    tma_load_4d(dst + kTileBytes + kHalfTile, mv, 64, g, t0, b, bar, pol);
  };
  int issued = 0;
  if (tid == 0) {
    for (; issued < kStages - 1 && issued < units; ++issued) {
      if (issued) next_unit<kRW, kKT>(a, ld);
      load_tile(ld, issued);
    }
  }

  uint32_t qf[kHD / 16][4];
  float o[kHD / 8][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
  int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;
  bool fresh = true, first_item = true;
  int stage = 0, it = 0;
  uint32_t phase = 0;
  for (; it < units; ++it) {
    const int grows = cp.u < 0 ? a.prows : a.rows;
    const int ra = cp.rt * kRW + gq, rb = ra + 8;   // this thread's two rows
    if (fresh) {
      const bool va = ra < grows, vb = rb < grows;
      const uint16_t *qa = a.q + q_row(a, cp.u, g, va ? ra : 0) * kHD + 2 * tq;
      const uint16_t *qb = a.q + q_row(a, cp.u, g, vb ? rb : 0) * kHD + 2 * tq;
#pragma unroll
      for (int kk = 0; kk < kHD / 16; ++kk) {
        qf[kk][0] = va ? *reinterpret_cast<const uint32_t *>(qa + 16 * kk) : 0u;
        qf[kk][1] = vb ? *reinterpret_cast<const uint32_t *>(qb + 16 * kk) : 0u;
        qf[kk][2] = va ? *reinterpret_cast<const uint32_t *>(qa + 16 * kk + 8) : 0u;
        qf[kk][3] = vb ? *reinterpret_cast<const uint32_t *>(qb + 16 * kk + 8) : 0u;
      }
#pragma unroll
      for (int d = 0; d < kHD / 8; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] = 0.0f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.0f;
      row_bounds(a, cp.u, cp.len, min(ra, grows - 1), lo0, hi0);
      row_bounds(a, cp.u, cp.len, min(rb, grows - 1), lo1, hi1);
      fresh = false;
    }
    bool ok = mbar_try_wait(full0 + 8 * stage, phase);
    if (!ok) ok = wait_bar(full0 + 8 * stage, phase, abort_flag, a.status);
    if (!__syncthreads_and(ok)) break;
    // every warp is done with the tile before this one: its stage takes the next load
    if (tid == 0 && issued < units) {
      if (issued) next_unit<kRW, kKT>(a, ld);
      load_tile(ld, stage == 0 ? kStages - 1 : stage - 1);
      ++issued;
    }
    const uint32_t kt = ring + stage * kStageBytes, vt = kt + kTileBytes;
    const int first_key = tile_key<kKT>(cp);
    const int sinks = cp.u < 0 ? 0 : a.sinks;
    if (first_key + kKT > cp.s.hi || (first_key < cp.s.lo && first_key + kKT > sinks)) {
      // value rows that no row sees: two threads a row, 64 dims each
      const int t = first_key + (tid >> 1);
      if (!(t < cp.s.hi && (t >= cp.s.lo || t < sinks))) {
        uint4 *row = reinterpret_cast<uint4 *>(sring + stage * kStageBytes + kTileBytes + (tid & 1) * kHalfTile +
                                               (tid >> 1) * 128);
#pragma unroll
        for (int c = 0; c < 8; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the stage's next load
      }
      __syncthreads();
    }

    const int t0 = first_key + 16 * warp;   // first key of this warp
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.0f;
      const uint32_t row = kt + (16 * warp + 8 * n + (lane & 7)) * 128;
#pragma unroll
      for (int kk = 0; kk < kHD / 16; kk += 2) {
        uint32_t b[4];
        ldsm4(row + (kk >> 2) * kHalfTile + ((((2 * kk + (lane >> 3)) & 7) ^ (lane & 7)) << 4), b);
        mma(s[n], qf[kk], b[0], b[1]);
        mma(s[n], qf[kk + 1], b[2], b[3]);
      }
    }
    // scores in log2 units; keys a row does not see become -inf
    const bool open = t0 >= lo0 && t0 >= lo1 && t0 + 16 <= hi0 && t0 + 16 <= hi1;
    float x0m = -INFINITY, x1m = -INFINITY;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int t = t0 + 8 * n + 2 * tq;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[n][i] *= a.scale_log2;
        s[n][2 + i] *= a.scale_log2;
        if (!open) {
          if (!(t + i < hi0 && (t + i >= lo0 || t + i < sinks))) s[n][i] = -INFINITY;
          if (!(t + i < hi1 && (t + i >= lo1 || t + i < sinks))) s[n][2 + i] = -INFINITY;
        }
        x0m = fmaxf(x0m, s[n][i]);
        x1m = fmaxf(x1m, s[n][2 + i]);
      }
    }
    if (kScored) {
      float *sa = a.smat + ((static_cast<int64_t>(cp.u) * a.nkv + g) * a.rows + ra) * a.s_ld;
      float *sb = sa + static_cast<int64_t>(8) * a.s_ld;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int t = t0 + 8 * n + 2 * tq;
        if (t < a.s_ld) {   // (s_ld is even)
          if (ra < grows) *reinterpret_cast<float2 *>(sa + t) = make_float2(s[n][0], s[n][1]);
          if (rb < grows) *reinterpret_cast<float2 *>(sb + t) = make_float2(s[n][2], s[n][3]);
        }
      }
    }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      x0m = fmaxf(x0m, __shfl_xor_sync(0xffffffffu, x0m, w));
      x1m = fmaxf(x1m, __shfl_xor_sync(0xffffffffu, x1m, w));
    }
    const float n0 = fmaxf(m0, x0m), n1 = fmaxf(m1, x1m);
    if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
      const float c0 = n0 > m0 ? ex2(m0 - n0) : 1.0f, c1 = n1 > m1 ? ex2(m1 - n1) : 1.0f;
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int d = 0; d < kHD / 8; ++d) {
        o[d][0] *= c0;
        o[d][1] *= c0;
        o[d][2] *= c1;
        o[d][3] *= c1;
      }
      m0 = n0;
      m1 = n1;
    }
    const float u0 = m0 == -INFINITY ? 0.0f : m0, u1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[n][i] = ex2(s[n][i] - u0);
        s[n][2 + i] = ex2(s[n][2 + i] - u1);
        l0 += s[n][i];
        l1 += s[n][2 + i];
      }
    }
    {
      uint32_t ph[4], pl[4];
      split2(s[0][0], s[0][1], ph[0], pl[0]);
      split2(s[0][2], s[0][3], ph[1], pl[1]);
      split2(s[1][0], s[1][1], ph[2], pl[2]);
      split2(s[1][2], s[1][3], ph[3], pl[3]);
      const uint32_t row = vt + (16 * warp + (lane & 15)) * 128;
#pragma unroll
      for (int d = 0; d < kHD / 16; ++d) {
        uint32_t b[4];
        ldsm4_t(row + (d >> 2) * kHalfTile + ((((2 * d + (lane >> 4)) & 7) ^ (lane & 7)) << 4), b);
        mma(o[2 * d], ph, b[0], b[1]);
        mma(o[2 * d + 1], ph, b[2], b[3]);
        mma(o[2 * d], pl, b[0], b[1]);
        mma(o[2 * d + 1], pl, b[2], b[3]);
      }
    }

    const bool item_end = cp.j == cp.s.n - 1;
    if (item_end || it == units - 1) {
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, w);
        l1 += __shfl_xor_sync(0xffffffffu, l1, w);
      }
      // join the warps, in the tile's own stage: the upper half of them hands its rows to
      // the lower, twice
      float *mrg = reinterpret_cast<float *>(sring + stage * kStageBytes);
#pragma unroll
      for (int half = 2; half > 0; half >>= 1) {
        __syncthreads();
        if (warp >= half && warp < 2 * half) {
          float *dst = mrg + (warp - half) * kMergeFloats;
#pragma unroll
          for (int d = 0; d < kHD / 8; ++d) {
            *reinterpret_cast<float2 *>(dst + gq * kHD + 8 * d + 2 * tq) = make_float2(o[d][0], o[d][1]);
            *reinterpret_cast<float2 *>(dst + (gq + 8) * kHD + 8 * d + 2 * tq) = make_float2(o[d][2], o[d][3]);
          }
          if (tq == 0) {
            dst[kRW * kHD + gq] = m0;
            dst[kRW * kHD + gq + 8] = m1;
            dst[kRW * kHD + 16 + gq] = l0;
            dst[kRW * kHD + 24 + gq] = l1;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncthreads();
        if (warp < half) {
          const float *src = mrg + warp * kMergeFloats;
          const float pm0 = src[kRW * kHD + gq], pm1 = src[kRW * kHD + gq + 8];
          const float pl0 = src[kRW * kHD + 16 + gq], pl1 = src[kRW * kHD + 24 + gq];
          const float w0 = fmaxf(m0, pm0), w1 = fmaxf(m1, pm1);
          const float z0 = w0 == -INFINITY ? 0.0f : w0, z1 = w1 == -INFINITY ? 0.0f : w1;
          const float a0 = ex2(m0 - z0), a1 = ex2(m1 - z1), b0 = ex2(pm0 - z0), b1 = ex2(pm1 - z1);
          l0 = l0 * a0 + pl0 * b0;
          l1 = l1 * a1 + pl1 * b1;
          m0 = w0;
          m1 = w1;
#pragma unroll
          for (int d = 0; d < kHD / 8; ++d) {
            const float2 s0 = *reinterpret_cast<const float2 *>(src + gq * kHD + 8 * d + 2 * tq);
            const float2 s1 = *reinterpret_cast<const float2 *>(src + (gq + 8) * kHD + 8 * d + 2 * tq);
            o[d][0] = o[d][0] * a0 + s0.x * b0;
            o[d][1] = o[d][1] * a0 + s0.y * b0;
            o[d][2] = o[d][2] * a1 + s1.x * b1;
            o[d][3] = o[d][3] * a1 + s1.y * b1;
          }
        }
      }
      if (warp == 0) {
        const bool whole = item_end && cp.item >= x0;
        float *po = nullptr;      // fp32 destination of rows ra, rb (null: out)
        float2 *pm = nullptr;
        int64_t ia = gq, ib = ia + 8;
        const int64_t qa = q_row(a, cp.u, g, ra), qb = q_row(a, cp.u, g, rb);
        if (!whole) {
          const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (first_item ? 0 : 1);
          po = a.part_o + slot * kRW * kHD;
          pm = a.part_ml + slot * kRW;
        } else if (a.P > 0) {
          const int64_t src = cp.u < 0 ? 0 : static_cast<int64_t>(a.B) * a.nr * a.nq;
          po = a.row_o + src * kHD;
          pm = a.row_ml + src;
          ia = qa;
          ib = qb;
        }
        if (po) {
#pragma unroll
          for (int d = 0; d < kHD / 8; ++d) {
            if (ra < grows)
              *reinterpret_cast<float2 *>(po + ia * kHD + 8 * d + 2 * tq) = make_float2(o[d][0], o[d][1]);
            if (rb < grows)
              *reinterpret_cast<float2 *>(po + ib * kHD + 8 * d + 2 * tq) = make_float2(o[d][2], o[d][3]);
          }
          if (tq == 0) {
            if (ra < grows) pm[ia] = make_float2(m0, l0);
            if (rb < grows) pm[ib] = make_float2(m1, l1);
          }
        } else {
          const float i0 = l0 > 0.0f ? 1.0f / l0 : 0.0f, i1 = l1 > 0.0f ? 1.0f / l1 : 0.0f;
#pragma unroll
          for (int d = 0; d < kHD / 8; ++d) {
            if (ra < grows)
              *reinterpret_cast<uint32_t *>(a.out + qa * kHD + 8 * d + 2 * tq) = pack_bf16(o[d][0] * i0, o[d][1] * i0);
            if (rb < grows)
              *reinterpret_cast<uint32_t *>(a.out + qb * kHD + 8 * d + 2 * tq) = pack_bf16(o[d][2] * i1, o[d][3] * i1);
          }
          if (kScored && tq == 0) {
            if (ra < grows) a.row_ml[qa] = make_float2(m0, i0);
            if (rb < grows) a.row_ml[qb] = make_float2(m1, i1);
          }
        }
      }
      fresh = true;
      first_item = false;
    }
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
    if (it + 1 < units) next_unit<kRW, kKT>(a, cp);
  }
  if (it < units && tid == 0) {   // gave up: let the copies already issued land before the CTA exits
    for (int j = it; j < issued; ++j) {
      const long long c0 = clock64();
      while (!mbar_try_wait(full0 + 8 * (j % kStages), static_cast<uint32_t>((j / kStages) & 1)) &&
             clock64() - c0 < kWaitCycles) {
      }
    }
  }
  wait_last(a);
}

// ------------------------------------------------------------------ plan
// Block 0 plans the launch a, block 1 (when the grid has it) the second one.
template <int RW, int KT, int PRW, int PKT>
__global__ void __launch_bounds__(kPlanThreads) ragged_plan_kernel(const __grid_constant__ Args a,
                                                                   const __grid_constant__ Args p) {
  pdl_wait();
  pdl_release();
  if (blockIdx.x == 0)
    make_plan<RW, KT>(a);
  else
    make_plan<PRW, PKT>(p);
}

// ------------------------------------------------------------------ joining the pieces
struct RowSum {
  float M, L, o[4];
  __device__ __forceinline__ void add(float2 ml, float4 v) {
    const float w = fmaxf(M, ml.x);
    const float z = w == -INFINITY ? 0.0f : w;
    const float x = ex2(M - z), y = ex2(ml.x - z);
    L = L * x + ml.y * y;
    o[0] = o[0] * x + v.x * y;
    o[1] = o[1] * x + v.y * y;
    o[2] = o[2] * x + v.z * y;
    o[3] = o[3] * x + v.w * y;
    M = w;
  }
};

// Where the pieces of a row lie: piece 0 at row `first` of o and ml, the others from row
// `second` on, `step` rows apart (a row that its range finished: its whole row).
struct Source {
  const float *o;
  const float2 *ml;
  int64_t first, second;
  int n, step;
};

// Row r_in of an item (row tiles of rw rows, kv head g), whole: row `whole` of row_o, row_ml.
__device__ __forceinline__ Source find_source(const float *part_o, const float2 *part_ml, int rw, int nkv, const Pieces &x,
                                              int g, int r_in, const float *row_o, const float2 *row_ml, int64_t whole) {
  Source s = {row_o, row_ml, whole, 0, x.n == 0 ? 0 : x.c1 - x.c0 + 1, 0};
  if (s.n > 1) {
    s.o = part_o;
    s.ml = part_ml;
    s.step = nkv * 2 * rw;
    const int64_t at = static_cast<int64_t>((x.c0 * nkv + g) * 2) * rw + r_in;   // (pieces are few)
    s.first = at + x.s0 * rw;
    s.second = at + s.step;
  }
  return s;
}

// Adds the pieces of p, then those of o, the loads of kBatch in flight together; of kSplit
// equal parts of them the one given.
template <int kBatch, int kSplit = 1>
__device__ __forceinline__ void add_pieces(const Source &p, const Source &o, int lane, RowSum &s, int part = 0) {
  const int all = p.n + o.n, n = all * (part + 1) / kSplit;
  for (int i0 = all * part / kSplit; i0 < n; i0 += kBatch) {
    float2 ml[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j;
      if (i < n) {
        const bool first = i < p.n;
        const Source &x = first ? p : o;
        const int k = first ? i : i - p.n;
        const int64_t at = k == 0 ? x.first : x.second + static_cast<int64_t>(k - 1) * x.step;
        ml[j] = __ldcg(x.ml + at);
        v[j] = __ldcg(reinterpret_cast<const float4 *>(x.o + at * kHD + 4 * lane));
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (i0 + j < n) s.add(ml[j], v[j]);
  }
}

__device__ __forceinline__ void store_row(const Args &a, int64_t row, int lane, const RowSum &s, bool scored) {
  const float inv = s.L > 0.0f ? 1.0f / s.L : 0.0f;
  *reinterpret_cast<uint2 *>(a.out + row * kHD + 4 * lane) =
      make_uint2(pack_bf16(s.o[0] * inv, s.o[1] * inv), pack_bf16(s.o[2] * inv, s.o[3] * inv));
  if (scored && lane == 0) a.row_ml[row] = make_float2(s.M, inv);
}

// The parts of a row that kSplit neighbouring warps added, joined in order by the first of
// them; by all threads of the CTA (8 warps).
template <int kSplit>
__device__ __forceinline__ void join_parts(RowSum &s, int lane, int part) {
  if (kSplit == 1) return;
  __shared__ float4 v[8][32];
  __shared__ float2 ml[8];
  const int warp = threadIdx.x >> 5;
  v[warp][lane] = make_float4(s.o[0], s.o[1], s.o[2], s.o[3]);
  if (lane == 0) ml[warp] = make_float2(s.M, s.L);
  __syncthreads();
  if (part == 0)
#pragma unroll
    for (int i = 1; i < kSplit; ++i) s.add(ml[warp + i], v[warp + i][lane]);
}

// A row's result is the sum over its pieces e^(m - M) o / sum e^(m - M) l, taken in order,
// one warp per row; items that one range held are finished already; the rows of row tiles
// without keys become zero.  kBatch: pieces of a row loaded together.  Bound by latency
// (with cold caches 4.4 us for 64 single tokens, 5 to 9 for one block; with a prefix 14 us
// at 32 x 8 queries of 40 heads, 32 to 35 at 192 x 8, which read 64 MB and more of fp32 rows and
// pieces).
//
// Few items (no more than ranges: spread over many of them, each batch of pieces a round trip
// to L2): CTA (item and kv head, 8 / kSplit rows), kSplit warps to a row.
template <int kBatch, int kSplit>
__global__ void __launch_bounds__(256) ragged_join_items_kernel(const __grid_constant__ Args a, int rw, int scored) {
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31;
  const int e = blockIdx.x / a.nkv, g = blockIdx.x - e * a.nkv;
  const Pieces f = a.direct ? request_pieces(warp_plan<kKT>(a, rw), e)
                            : load_pieces(a.pieces + a.PRT + e);
  if (f.n > 0 && f.c0 == f.c1) return;
  const int warp = threadIdx.x >> 5, part = warp % kSplit;
  const int b = e / a.RT, r_in = blockIdx.y * (8 / kSplit) + warp / kSplit, r = (e - b * a.RT) * rw + r_in;
  const bool in = r_in < rw && r < a.rows;
  RowSum s = {-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
  const Source none = {nullptr, nullptr, 0, 0, 0, 0};
  if (in)
    add_pieces<kBatch, kSplit>(find_source(a.part_o, a.part_ml, rw, a.nkv, f, g, r_in, nullptr, nullptr, 0), none, lane, s,
                               part);
  join_parts<kSplit>(s, lane, part);
  if (in && part == 0) store_row(a, q_row(a, b, g, r), lane, s, scored);
}

// Many items: CTA (range and kv head, `per` rows): the item that begins in the range and goes
// on in the next, if there is one.  The last block row of the grid zeroes the rows without
// keys, each range looking through its share of the requests.
template <int kBatch>
__global__ void __launch_bounds__(256) ragged_join_kernel(const __grid_constant__ Args a, int rw, int per, int scored) {
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int range = blockIdx.x / a.nkv, g = blockIdx.x - range * a.nkv;
  if (blockIdx.y == gridDim.y - 1) {
    if (!__ldcg(&a.plan->empty)) return;
    for (int b = range; b < a.B; b += a.groups)
      for (int rt = 0; rt < a.RT; ++rt) {
        if (__ldcg(&a.pieces[a.PRT + b * a.RT + rt].n)) continue;
        const RowSum s = {-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
        for (int r = rt * rw + warp; r < min((rt + 1) * rw, a.rows); r += 8) store_row(a, q_row(a, b, g, r), lane, s, scored);
      }
    return;
  }
  if (range + 1 >= __ldcg(&a.plan->ranges)) return;
  const int x0 = __ldcg(a.begins + range);
  const Place p = load_place(a, a.places + range + 1);   // its item goes on in the next range ...
  if (p.j == 0 || p.item < x0) return;                   // ... and begins in this one
  const Pieces f = load_pieces(a.pieces + a.PRT + p.u * a.RT + p.rt);
  for (int r_in = blockIdx.y * per + warp; r_in < (static_cast<int>(blockIdx.y) + 1) * per; r_in += 8) {
    const int r = p.rt * rw + r_in;
    if (r_in >= rw || r >= a.rows) return;
    RowSum s = {-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
    const Source none = {nullptr, nullptr, 0, 0, 0, 0};
    add_pieces<kBatch>(find_source(a.part_o, a.part_ml, rw, a.nkv, f, g, r_in, nullptr, nullptr, 0), none, lane, s);
    store_row(a, q_row(a, p.u, g, r), lane, s, scored);
  }
}

// With a prefix every row joins its prefix's and its request's results.  CTA (`per` rows of a
// request's kv head), kSplit warps per row at a time (then per = 8 / kSplit).
template <int kBatch, int kSplit>
__global__ void __launch_bounds__(256, kBatch == 4 ? 4 : 1) ragged_join_prefix_kernel(const __grid_constant__ Args a, int rw, int per) {
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31;
  const int chunks = (a.rows + per - 1) / per, bg = blockIdx.x / chunks;
  const int b = bg / a.nkv, g = bg - b * a.nkv;
  const int r0 = (blockIdx.x - bg * chunks) * per, r1 = min(r0 + per, a.rows);
  const int prw = a.pre.rw;
  const int64_t nrow = static_cast<int64_t>(a.B) * a.nr * a.nq;
  WarpPlan w = {};
  if (a.direct) w = warp_plan<kKT>(a, rw);
  const int warp = threadIdx.x >> 5, part = warp % kSplit;
  for (int rr = r0 + warp / kSplit; kSplit > 1 || rr < r1; rr += 8) {
    const int r = min(rr, r1 - 1);   // (kSplit > 1: one round, which all warps make)
    const int R = b * a.rows + r, pt = R / prw, t = r / rw;
    const Pieces fp = a.direct ? prefix_pieces(w, pt) : load_pieces(a.pre.pieces + pt);
    const Pieces fo = a.direct ? request_pieces(w, b * a.RT + t) : load_pieces(a.pieces + a.PRT + b * a.RT + t);
    const int64_t row = q_row(a, b, g, r);
    RowSum s = {-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
    add_pieces<kBatch, kSplit>(
        find_source(a.pre.part_o, a.pre.part_ml, prw, a.nkv, fp, g, R - pt * prw, a.row_o, a.row_ml, row),
        find_source(a.part_o, a.part_ml, rw, a.nkv, fo, g, r - t * rw, a.row_o, a.row_ml, nrow + row), lane, s, part);
    join_parts<kSplit>(s, lane, part);
    if (part == 0 && r == rr) store_row(a, row, lane, s, false);
    if (kSplit > 1) return;
  }
}

// ------------------------------------------------------------------ column sums
// scores_out[b, g, t] = decay * scores_in[b, g, t] + sum over the group's rows of the
// weight e^(s - M) / L, t < len, from the row scores that the decode kernel left (at most
// 64 bytes a key and kv head: in L2 still at the sizes below, 15 MB; more than 129 MB of them
// come from memory); rows in order.  CTA (2048 keys of a kv head: with 512, most
// of the time went by in CTAs behind the requests' ends), a thread's four key pairs together
// (one after the other they waited for each other's loads: 32 requests of 8 kv heads and 93
// thousand keys, 5 rows, 16.6 us; together 10.8).
constexpr int kColumnKeys = 2048;
__global__ void __launch_bounds__(256) ragged_columns_kernel(const __grid_constant__ Args a) {
  __shared__ float2 ml[kRW];
  pdl_wait();
  pdl_release();
  const int chunks = (a.cache_len + kColumnKeys - 1) / kColumnKeys, bg = blockIdx.x / chunks;
  const int chunk = blockIdx.x - bg * chunks, b = bg / a.nkv, g = bg % a.nkv;
  const int len = clamp_len(a, b), end = min(len, (chunk + 1) * kColumnKeys);
  if (chunk * kColumnKeys >= len) return;
  if (static_cast<int>(threadIdx.x) < a.rows) {
    const float2 x = a.row_ml[q_row(a, b, g, threadIdx.x)];
    ml[threadIdx.x] = x.x == -INFINITY ? make_float2(0.0f, 0.0f) : x;
  }
  __syncthreads();
  // key pairs t0 + 512 i, all of them together
  constexpr int kPairs = kColumnKeys / 512;
  const int t0 = chunk * kColumnKeys + 2 * threadIdx.x;
  const float *s = a.smat + static_cast<int64_t>(bg) * a.rows * a.s_ld + t0;
  const int64_t at = static_cast<int64_t>(bg) * a.cache_len + t0;
  float in[kPairs][2], w[kPairs][2];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    w[i][0] = w[i][1] = 0.0f;
    in[i][0] = a.scores_in && t0 + 512 * i < end ? a.scores_in[at + 512 * i] : 0.0f;
    in[i][1] = a.scores_in && t0 + 512 * i + 1 < end ? a.scores_in[at + 512 * i + 1] : 0.0f;
  }
  const int64_t ld = a.s_ld;
#pragma unroll 4
  for (int r = 0; r < a.rows; ++r) {
    float2 v[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      if (t0 + 512 * i < end) v[i] = __ldcs(reinterpret_cast<const float2 *>(s + r * ld + 512 * i));
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      w[i][0] += ex2(v[i].x - ml[r].x) * ml[r].y;
      w[i][1] += ex2(v[i].y - ml[r].x) * ml[r].y;
    }
  }
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    if (t0 + 512 * i < end) a.scores_out[at + 512 * i] = __fmaf_rn(a.decay, in[i][0], w[i][0]);
    if (t0 + 512 * i + 1 < end) a.scores_out[at + 512 * i + 1] = __fmaf_rn(a.decay, in[i][1], w[i][1]);
  }
}

template <int RW, int KT, int PRW, int PKT>
cudaError_t launch_plan(const Args &a, const Args *p, cudaStream_t stream) {
  return launch_pdl(ragged_plan_kernel<RW, KT, PRW, PKT>, dim3(p ? 2 : 1), dim3(kPlanThreads), 0, stream, a, p ? *p : a);
}

}  // namespace

dspark_status_t plan_launch(const Args &a, Form form, const Args *p, Kind kind, cudaStream_t stream) {
  constexpr int MR = kMmaRows, MK = kMmaKeys, SR = kStreamRows, R = kSharedRows, K = kTcKeys;
  const cudaError_t e = form == kMma       ? launch_plan<MR, MK, R, K>(a, p, stream)
                        : form == kShared  ? launch_plan<R, K, R, K>(a, p, stream)
                        : kind == kScored  ? launch_plan<SR, K, SR, kWeightKeys>(a, p, stream)
                                           : launch_plan<SR, K, R, K>(a, p, stream);
  if (e != cudaSuccess) return DSPARK_ERR_CUDA;
  count_launches(1);
  return DSPARK_OK;
}

dspark_status_t mma_launch(const Args &a, bool scored, cudaStream_t stream) {
  MmaParams prm;
  prm.a = a;
  if (!cache_map(&prm.k, a.k_cache, a.B, a.cache_len, a.nkv, kKT) ||
      !cache_map(&prm.v, a.v_cache, a.B, a.cache_len, a.nkv, kKT))
    return DSPARK_ERR_UNSUPPORTED_SHAPE;
  prm.kp = prm.k;
  prm.vp = prm.v;
  if (a.PRT > 0 && (!cache_map(&prm.kp, a.k_prefix, 1, a.P, a.nkv, kKT) || !cache_map(&prm.vp, a.v_prefix, 1, a.P, a.nkv, kKT)))
    return DSPARK_ERR_UNSUPPORTED_SHAPE;
  auto kern = scored ? ragged_mma_kernel<true> : ragged_mma_kernel<false>;
  static std::atomic<bool> done[2][64];
  if (!allow_smem(kern, kSmem, done[scored])) return DSPARK_ERR_CUDA;
  if (launch_pdl(kern, dim3(static_cast<unsigned>(a.groups * a.nkv)), dim3(kThreads), kSmem, stream, prm) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  count_launches(1);
  return DSPARK_OK;
}

dspark_status_t join_launch(const Args &a, int rw, bool scored, cudaStream_t stream) {
  // four warps to a row where it may have more pieces than one loads together (4 tokens over a
  // prefix of 4096 3 us less, a scored block over 2057 keys 2 us less; with 9 pieces, a block
  // with a window of 512, 1.2 us more: not there)
  constexpr int kSplit = 4, kBatch = 16;
  cudaError_t e;
  if (a.P > 0) {
    // the prefix's items are cut into about groups / items pieces; 8 rows (one per warp) per
    // CTA, 64 where that still fills the GPU
    const int items = (a.prows + a.pre.rw - 1) / a.pre.rw;
    const bool split = a.pre.groups > 4 * items && a.P > kBatch * kKT;
    const int per = split ? 8 / kSplit : a.prows * static_cast<long long>(a.nkv) > 32768 ? 64 : 8;
    const dim3 grid(static_cast<unsigned>(a.B) * a.nkv * ((a.rows + per - 1) / per));
    e = launch_pdl(split                       ? ragged_join_prefix_kernel<kBatch, kSplit>
                   : a.pre.groups <= 4 * items ? ragged_join_prefix_kernel<4, 1>
                                               : ragged_join_prefix_kernel<kBatch, 1>,
                   grid, dim3(256), 0, stream, a, rw, per);
  } else {
    const int in_tile = a.rows < rw ? a.rows : rw, items = a.B * a.RT;
    if (items <= a.groups) {
      const long long seen = static_cast<long long>(a.window) + a.nr + a.sinks;
      const long long keys = a.window > 0 && seen < a.cache_len ? seen : a.cache_len;
      const bool split = a.groups > kBatch * items && keys > kBatch * kKT;
      const int per = split ? 8 / kSplit : 8;
      const dim3 grid(static_cast<unsigned>(items * a.nkv), static_cast<unsigned>((in_tile + per - 1) / per));
      e = launch_pdl(split ? ragged_join_items_kernel<kBatch, kSplit> : ragged_join_items_kernel<kBatch, 1>, grid, dim3(256), 0,
                     stream, a, rw, scored ? 1 : 0);
    } else {
      // up to 64 rows one per warp, else four: a piece's rows are joined by up to 8 CTAs
      const int per = in_tile > 64 ? 32 : 8;
      const dim3 grid(static_cast<unsigned>(a.groups * a.nkv), static_cast<unsigned>((in_tile + per - 1) / per + 1));
      e = launch_pdl(ragged_join_kernel<4>, grid, dim3(256), 0, stream, a, rw, per, scored ? 1 : 0);
    }
  }
  if (e != cudaSuccess) return DSPARK_ERR_CUDA;
  count_launches(1);
  return DSPARK_OK;
}

dspark_status_t columns_launch(const Args &a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.nkv * ((a.cache_len + kColumnKeys - 1) / kColumnKeys));
  if (launch_pdl(ragged_columns_kernel, grid, dim3(256), 0, stream, a) != cudaSuccess) return DSPARK_ERR_CUDA;
  count_launches(1);
  return DSPARK_OK;
}

}  // namespace ragged
}  // namespace dspark
