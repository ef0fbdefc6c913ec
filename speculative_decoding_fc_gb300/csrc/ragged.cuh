// Attention over key/value caches whose requests differ in length: the arguments, the
// masks and the work schedule shared by its kernels.
//
// Rows and groups.  A query row is one (query, head) pair; the rows that read the same
// keys form a group: for request b and kv head g the nr * grp rows (r = i * grp + hh,
// query i, head g * grp + hh, grp = nq / nkv).  With a shared prefix all requests' rows
// of a kv head form one more group, B * nr * grp rows over the prefix keys.  Group index
// u: the prefix (when there is one) is u = 0 and request b is u = b + has_prefix.
//
// Masks.  Row i of a request of len keys stands at position p = len - nr + i and sees
// key t iff t < len, (t < sinks or t > p - window; no window: every t) and, when causal,
// t <= p.  A row may see no key at all: its output is zero.
//
// Schedule.  A group's rows are cut into tiles of RW rows and their keys into tiles of KT
// keys; a (group, row tile) is an item and each of its key tiles one unit.  The units of
// all items, in the order (u, row tile, key tile), are cut into ranges of equal cost, so that
// the CTAs carry the same load however the lengths differ: an item costs its units and three
// more, the time to change to it (without them a CTA with six short requests took twice as
// long as one with a part of a long one).  A range is taken by nkv
// neighbouring CTAs, one per kv head, which pass over the same keys at about the same time:
// a key's heads are neighbours in memory (nkv * 256 bytes), and one CTA alone would leave
// the DRAM pages it opens to be opened again for every other head.  ragged_plan_kernel
// works the ranges out from the lengths on the device (a captured graph follows them); the
// other kernels read where their range begins.  (Each CTA finding its own place took 3 to 8
// us of dependent loads and shuffles, the plan kernel about 3 us once, 6 with cold caches.)  Up to 32 items each
// warp that needs its range has one lane per item work it out instead (WarpPlan) and the plan's
// launch is left out: one draft block over 1032 keys took 2.4 us less, 32 single tokens 74.2 ->
// 71.8.
// An item held by one range is finished there; every other item leaves pieces
// (unnormalised fp32 output, row maximum and sum), at most two per range and head (the
// range's first and last item), which a last kernel joins in range order: results do not
// depend on timing.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "ragged_host.h"

namespace dspark {
namespace ragged {

constexpr int kHD = 128;

// The keys of one row tile: those below hi that are at least lo or below sinks.  Key
// tile j of the item starts at key KT * j for j < sk (tiles of sinks in front of the
// window's first tile), else at KT * (lo_t + j - sk).
struct Span {
  int n;            // key tiles
  int sk, lo_t;
  int lo, hi;       // item-wide bounds (the union over the tile's rows)
};

// A place in the unit order.
struct __align__(16) Place {
  Span s;
  int u;            // -1: the prefix group, else the request
  int rt, j;
  int len;
  int item;         // first unit of the item
  int next_len;     // of the next request (loaded ahead by the kernels that walk on)
};

// Where an item's results lie: its pieces in ranges c0 .. c1 (the first in its range's
// slot s0, the others in slot 0: their ranges begin inside the item), or the item's own
// rows when one range held it.
struct __align__(16) Pieces {
  int n;            // key tiles of the item (0: nothing)
  int c0, c1, s0;
};

struct __align__(16) Plan {
  int total;        // units
  int ranges;       // in use: at most the launch's groups, never more than there are units
  int empty;        // some request has a row tile without keys
  int pad;
};

// Where the prefix's results lie: those of this launch or of one of its own.
struct PrefixSource {
  const Pieces *pieces;                 // of the prefix's row tiles
  const float *part_o;
  const float2 *part_ml;
  int rw;                               // rows per row tile
  int groups;                           // of its launch
};

struct Args {
  const uint16_t *q;                    // [B, nr, nq, 128]
  const uint16_t *k_cache, *v_cache;    // [B, cache_len, nkv, 128]
  const uint16_t *k_prefix, *v_prefix;  // [P, nkv, 128] (P > 0)
  const int32_t *lens;                  // [B]
  uint16_t *out;                        // [B, nr, nq, 128]
  Plan *plan;
  Place *places;                        // [groups]: where range c begins
  int *begins;                          // [groups + 1]: its first unit, then the total
  int2 *bases;                          // [sB * RT + 1]: first unit of each item of a request (and the items with
                                        // keys before it), then the total
  Pieces *pieces;                       // [PRT + sB * RT]: of the prefix's items, then of the requests' 
  float *part_o;                        // pieces [groups * nkv * 2][RW][128]
  float2 *part_ml;                      // [groups * nkv * 2][RW]: row maximum (log2 units) and sum
  float *row_o;                         // prefix: whole items' rows [2][B * nr * nq][128] (0 prefix, 1 own keys)
  float2 *row_ml;                       // prefix: [2][B * nr * nq]; scored: [B * nr * nq] (maximum, 1 / sum)
  PrefixSource pre;
  float *smat;                          // scored, decode kernel: row scores [B * nkv][rows][s_ld] (log2 units)
  const float *scores_in;               // scored: [B, nkv, cache_len] or null
  float *scores_out;
  float decay;
  int s_ld;
  int B, nr, nq, nkv, grp, cache_len, P;
  int window, sinks, causal;            // window 0: none
  int rows, RT, prows, PRT;             // rows and row tiles of a request's group and of the prefix's
  int sB;                               // requests in the launch's schedule (B, or 0: the prefix alone)
  int groups;                           // ranges the launch has CTAs for
  int direct;                           // no plan: every warp works its range out itself (WarpPlan)
  int late_wait;                        // the launch before is the prefix's own (wait_first, wait_last)
  int ordinary;                         // this launch starts when everything before it has ended
  float scale_log2;                     // log2(e) / sqrt(128)
  int *status;
};

// The launch over the own keys after one over the prefix reads nothing of that one's and does
// not wait for it: it fills the SMs that the prefix's last CTAs leave.  What it does read (the
// plan, q, the lengths, the caches) it may read without a wait of its own because the prefix's
// launch is an ordinary one: that grid starts when everything before it in the stream has ended,
// with its writes visible to whatever starts later, and a programmatic launch overlaps with the
// one launch before it only.  (Behind a programmatic launch of the prefix it would rest on that
// grid's waits, which promise visibility to that grid alone.)  It ends behind the prefix's
// launch, so that the join, which waits for this launch, finds both complete.  32 x 8
// queries over a prefix of 16384: 108 us -> 101 (the ordinary launch costs 1 of them).
__device__ __forceinline__ void wait_first(const Args &a) {
  if (!a.late_wait) pdl_wait();
}
__device__ __forceinline__ void wait_last(const Args &a) {
  if (a.late_wait) pdl_wait();
}

__device__ __forceinline__ int clamp_len(const Args &a, int b) {
  const int n = __ldcg(a.lens + b);
  return n < 0 ? 0 : (n > a.cache_len ? a.cache_len : n);
}

template <int KT>
__device__ __forceinline__ Span make_span(int lo, int hi, int sinks) {
  Span s;
  s.lo = lo;
  s.hi = hi;
  s.lo_t = lo / KT;
  const int hi_t = hi > lo ? (hi + KT - 1) / KT : s.lo_t;
  const int sk_keys = sinks < hi ? sinks : hi;
  const int sk_t = (sk_keys + KT - 1) / KT;
  s.sk = sk_t < s.lo_t ? sk_t : s.lo_t;
  s.n = s.sk + hi_t - s.lo_t;
  return s;
}

// Row tile rt (of rw rows) of a request group of length len.
template <int KT>
__device__ __forceinline__ Span request_span(const Args &a, int rw, int len, int rt) {
  const int i0 = rt * rw / a.grp;
  const int rl = min((rt + 1) * rw, a.rows) - 1;
  const int p0 = len - a.nr + i0, p1 = len - a.nr + rl / a.grp;
  int hi = a.causal ? min(len, p1 + 1) : len;
  if (hi < 0) hi = 0;
  int lo = a.window > 0 ? p0 - a.window + 1 : 0;
  if (lo < 0) lo = 0;
  if (lo > hi) lo = hi;
  return make_span<KT>(lo, hi, a.sinks);
}

// Moves to the next row tile or group that has units (there is one).
template <int RW, int KT>
__device__ __forceinline__ void next_item(const Args &a, Place &p) {
  p.item += p.s.n;
  do {
    if (++p.rt == (p.u < 0 ? a.PRT : a.RT)) {
      p.rt = 0;
      if (++p.u >= a.sB) {   // past the last unit: nothing reads this place
        p.s.n = 0x7fffffff;
        return;
      }
      p.len = p.next_len;
      if (p.u + 1 < a.sB) p.next_len = clamp_len(a, p.u + 1);
    }
    p.s = p.u < 0 ? make_span<KT>(0, a.P, 0) : request_span<KT>(a, RW, p.len, p.rt);
  } while (p.s.n == 0);
  p.j = 0;
}

template <int RW, int KT>
__device__ __forceinline__ void next_unit(const Args &a, Place &p) {
  if (++p.j == p.s.n) next_item<RW, KT>(a, p);
}

// First key of the place's tile.
template <int KT>
__device__ __forceinline__ int tile_key(const Place &p) {
  return KT * (p.j < p.s.sk ? p.j : p.s.lo_t + p.j - p.s.sk);
}

// The plan of a launch, by one CTA (kPlanThreads threads).
constexpr int kPlanThreads = 512;
constexpr int kPlanItems = 2048;   // items whose first units are also kept in shared memory
constexpr int kItemCost = 3;       // units
template <int RW, int KT>
__device__ void make_plan(const Args &a) {
  __shared__ int2 s_base[kPlanItems];
  __shared__ int2 s_warp[kPlanThreads / 32];
  __shared__ int2 s_carry;
  __shared__ int s_empty, s_begins[kMaxRanges];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pn = (a.P + KT - 1) / KT, pre = a.PRT * pn;
  const int items = a.sB * a.RT;
  if (tid == 0) {
    s_carry = make_int2(pre, a.PRT);
    s_empty = 0;
  }
  __syncthreads();
  for (int e0 = 0; e0 < items; e0 += kPlanThreads) {
    const int e = e0 + tid;
    int n = 0;
    if (e < items) {
      const int b = e / a.RT, raw = __ldcg(a.lens + b);
      if (raw < 0 || raw > a.cache_len) record_error(a.status, DSPARK_ERR_INVALID_ARG);
      n = request_span<KT>(a, RW, raw < 0 ? 0 : min(raw, a.cache_len), e - b * a.RT).n;
      if (n == 0) s_empty = 1;
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    const unsigned some = __ballot_sync(0xffffffffu, n > 0);
    const int before = __popc(some & ((1u << lane) - 1u));
    if (lane == 31) s_warp[warp] = make_int2(inc, __popc(some));
    __syncthreads();
    int2 base = s_carry;
    for (int w = 0; w < warp; ++w) {
      base.x += s_warp[w].x;
      base.y += s_warp[w].y;
    }
    if (e < items) {
      const int2 at = make_int2(base.x + inc - n, base.y + before);
      a.bases[e] = at;
      if (e < kPlanItems) s_base[e] = at;
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) s_carry = make_int2(base.x + inc, base.y + before + (n > 0 ? 1 : 0));
    __syncthreads();
  }
  const int2 end = s_carry;
  const int ranges = min(a.groups, end.x);
  // few units: each its own range, or nearly so
  const int extra = end.x >= 2 * kItemCost * a.groups ? kItemCost : 0;
  const long long cost = end.x + static_cast<long long>(end.y) * extra;
  if (tid == 0) {
    a.plan->total = end.x;
    a.plan->ranges = ranges;
    a.plan->empty = s_empty;
    a.bases[items] = end;
    a.begins[ranges] = end.x;
  }
  for (int c = tid; c < ranges; c += kPlanThreads) {
    const long long x = cost * c / ranges;   // each range's cost exceeds `extra`: it holds a unit
    const long long pre_cost = static_cast<long long>(a.PRT) * (pn + extra);
    Place at;
    long long j;
    if (x < pre_cost) {
      at.u = -1;
      at.len = 0;
      at.s = make_span<KT>(0, a.P, 0);
      at.rt = static_cast<int>(x / (pn + extra));
      at.item = at.rt * pn;
      j = x - static_cast<long long>(at.rt) * (pn + extra);
    } else {
      int lo = 0, hi = items;   // the last item that begins at or before x
      int2 base = make_int2(pre, a.PRT);
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        const int2 v = mid < kPlanItems ? s_base[mid] : __ldcg(a.bases + mid);
        if (v.x + static_cast<long long>(v.y) * extra <= x) {
          lo = mid;
          base = v;
        } else {
          hi = mid;
        }
      }
      at.u = lo / a.RT;
      at.rt = lo - at.u * a.RT;
      at.len = clamp_len(a, at.u);
      at.s = request_span<KT>(a, RW, at.len, at.rt);
      at.item = base.x;
      j = x - base.x - static_cast<long long>(base.y) * extra;
    }
    at.j = j > extra ? static_cast<int>(j) - extra : 0;
    a.places[c] = at;
    a.begins[c] = s_begins[c] = at.item + at.j;
  }
  __syncthreads();
  auto range_of = [&](int x) {   // the range that holds unit x
    int lo = 0, hi = ranges;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s_begins[mid] <= x)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };
  auto base_of = [&](int e) { return e < min(items, kPlanItems) ? s_base[e].x : __ldcg(&a.bases[e].x); };
  for (int e = tid - a.PRT; e < items; e += kPlanThreads) {
    const int x = e < 0 ? (e + a.PRT) * pn : base_of(e);
    Pieces f = {e < 0 ? pn : base_of(e + 1) - x, 0, 0, 0};
    if (f.n > 0) {
      f.c0 = range_of(x);
      f.c1 = range_of(x + f.n - 1);
      f.s0 = s_begins[f.c0] == x ? 0 : 1;
    }
    a.pieces[a.PRT + e] = f;
  }
}

__device__ __forceinline__ Pieces load_pieces(const Pieces *at) {
  const int4 v = __ldcg(reinterpret_cast<const int4 *>(at));
  return {v.x, v.y, v.z, v.w};
}
__device__ __forceinline__ Place load_place(const Args &a, const Place *at) {
  Place p;
  const int4 *src = reinterpret_cast<const int4 *>(at);
  const int4 x = __ldcg(src), y = __ldcg(src + 1), z = __ldcg(src + 2);
  p.s.n = x.x;
  p.s.sk = x.y;
  p.s.lo_t = x.z;
  p.s.lo = x.w;
  p.s.hi = y.x;
  p.u = y.y;
  p.rt = y.z;
  p.j = y.w;
  p.len = z.x;
  p.item = z.y;
  p.next_len = p.u + 1 < a.sB ? clamp_len(a, p.u + 1) : 0;
  return p;
}

// The schedule of at most 32 items of requests, item e in lane e: the values that make_plan
// writes, in closed form.  The host takes this way only where the units' cost times the
// ranges fits 32 bits (64-bit divisions cost the joins 6 us).
constexpr int kDirectItems = 32;
struct WarpPlan {
  int n, len, base;         // this lane's item: units, the request's length, first unit
  uint32_t at;              // the cost before it
  int pn;                   // units of a row tile of the prefix
  int items, total;
  uint32_t ranges, extra, cost;
};

// By a whole warp; row tiles of rw rows.
template <int KT>
__device__ __forceinline__ WarpPlan warp_plan(const Args &a, int rw) {
  const int lane = threadIdx.x & 31;
  WarpPlan w;
  w.items = a.sB * a.RT;
  w.pn = (a.P + KT - 1) / KT;
  w.n = w.len = 0;
  if (lane < w.items) {
    const int b = lane / a.RT;
    w.len = clamp_len(a, b);
    w.n = request_span<KT>(a, rw, w.len, lane - b * a.RT).n;
  }
  int inc = w.n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  const unsigned some = __ballot_sync(0xffffffffu, w.n > 0);
  w.base = a.PRT * w.pn + inc - w.n;
  w.total = a.PRT * w.pn + __shfl_sync(0xffffffffu, inc, 31);
  w.ranges = min(a.groups, w.total);
  w.extra = w.total >= 2 * kItemCost * a.groups ? kItemCost : 0;
  w.at = w.base + (a.PRT + __popc(some & ((1u << lane) - 1u))) * w.extra;
  w.cost = w.total + (a.PRT + __popc(some)) * w.extra;
  return w;
}

// Range c of the launch: its first unit and the units in it; 0 units: no such range.
template <int RW, int KT>
__device__ __forceinline__ void find_range(const Args &a, int c, Place &p, int &x0, int &units) {
  units = 0;
  if (!a.direct) {
    if (c >= __ldcg(&a.plan->ranges)) return;
    x0 = __ldcg(a.begins + c);
    units = __ldcg(a.begins + c + 1) - x0;
    p = load_place(a, a.places + c);
    return;
  }
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && static_cast<int>(threadIdx.x) < a.sB) {
    const int raw = __ldcg(a.lens + threadIdx.x);
    if (raw < 0 || raw > a.cache_len) record_error(a.status, DSPARK_ERR_INVALID_ARG);
  }
  const WarpPlan w = warp_plan<KT>(a, RW);
  if (c >= static_cast<int>(w.ranges)) return;
  // the item (below 0: of the prefix), and the tile in it, where range r begins
  auto locate = [&](int r, int &e, int &item, int &j) {
    const uint32_t x = w.cost * r / w.ranges;
    uint32_t off;
    if (x < a.PRT * (w.pn + w.extra)) {
      const int rt = x / (w.pn + w.extra);
      e = rt - a.PRT;
      item = rt * w.pn;
      off = x - rt * (w.pn + w.extra);
    } else {
      e = 31 - __clz(__ballot_sync(0xffffffffu, lane < w.items && w.at <= x));
      item = __shfl_sync(0xffffffffu, w.base, e);
      off = x - __shfl_sync(0xffffffffu, w.at, e);
    }
    j = off > w.extra ? off - w.extra : 0;
  };
  int e, item, j, end = w.total;
  if (c + 1 < static_cast<int>(w.ranges)) {
    locate(c + 1, e, item, j);
    end = item + j;
  }
  locate(c, e, item, j);
  x0 = item + j;
  units = end - x0;
  p.item = item;
  p.j = j;
  if (e < 0) {
    p.u = -1;
    p.rt = e + a.PRT;
    p.len = 0;
    p.s = make_span<KT>(0, a.P, 0);
  } else {
    p.u = e / a.RT;
    p.rt = e - p.u * a.RT;
    p.len = __shfl_sync(0xffffffffu, w.len, e);
    p.s = request_span<KT>(a, RW, p.len, p.rt);
  }
  p.next_len = __shfl_sync(0xffffffffu, w.len, min(31, (p.u + 1) * a.RT));
}

// The pieces of an item of n units with the cost `at` before it (uniform over the warp): a
// range begins at or before a unit iff its cost is at most the unit's.
__device__ __forceinline__ Pieces find_pieces(const WarpPlan &w, int n, uint32_t at) {
  Pieces f = {n, 0, 0, 0};
  if (n > 0) {
    f.c0 = ((at + w.extra + 1) * w.ranges - 1) / w.cost;
    f.c1 = ((at + w.extra + n) * w.ranges - 1) / w.cost;
    f.s0 = w.cost * f.c0 / w.ranges >= at ? 0 : 1;
  }
  return f;
}
__device__ __forceinline__ Pieces request_pieces(const WarpPlan &w, int e) {
  return find_pieces(w, __shfl_sync(0xffffffffu, w.n, e), __shfl_sync(0xffffffffu, w.at, e));
}
__device__ __forceinline__ Pieces prefix_pieces(const WarpPlan &w, int rt) {
  return find_pieces(w, w.pn, rt * (w.pn + w.extra));
}

// Row r of group u and kv head g: its row of q and out ([B * nr * nq, 128]).
__device__ __forceinline__ int64_t q_row(const Args &a, int u, int g, int r) {
  const int i = r / a.grp;
  return (static_cast<int64_t>(u < 0 ? 0 : u) * a.nr + i) * a.nq + g * a.grp + (r - i * a.grp);
}

// The keys row r of request length len sees: t < hi and (t >= lo or t < sinks).
__device__ __forceinline__ void row_bounds(const Args &a, int u, int len, int r, int &lo, int &hi) {
  if (u < 0) {
    lo = 0;
    hi = a.P;
    return;
  }
  const int p = len - a.nr + r / a.grp;
  lo = a.window > 0 ? p - a.window + 1 : 0;
  hi = a.causal ? min(len, p + 1) : len;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 rounded to bf16, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *map, int x, int y, int z, int w, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}

}  // namespace ragged
}  // namespace dspark
