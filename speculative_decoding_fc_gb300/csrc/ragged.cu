// Host side of the ragged-cache attention calls: workspace layout and kernel choice.
#include <algorithm>
#include <cmath>

#include "ragged.cuh"
#include "ragged_host.h"
#include "tcgen05.cuh"

namespace dspark {
namespace ragged {
namespace {

// The kernel for groups of so many query rows per kv head.  Up to 16 rows one warp-level
// MMA's height holds them and the decode kernel waits for memory only; at 40 rows (the
// draft block of 8 tokens, 5 heads a group) the same kernel spent 3700 cycles of products
// per 64 keys that take 1400 to read.  Up to 64 rows the tcgen05 kernel's two halves read
// keys of their own, their reading the bound; more rows share each key tile.
Form form_of(long long rows) { return rows <= kMmaRows ? kMma : (rows <= kStreamRows ? kStreams : kShared); }

int tile_rows(Form f) { return f == kMma ? kMmaRows : (f == kStreams ? kStreamRows : kSharedRows); }
int tile_keys(Form f) { return f == kMma ? kMmaKeys : kTcKeys; }

// Ranges of a launch's schedule: two to an SM, one in the shared form (more CTAs than fit
// at once only when there are more kv heads than that).
int range_count(Form f, int sms, int nkv) {
  const int per_head = (f == kShared ? 1 : 2) * sms / nkv;
  return per_head > 0 ? per_head : 1;
}

static_assert(2 * kMaxGemmCtas <= kMaxRanges, "a schedule's ranges");

size_t piece_rows(Form f, int nkv) {
  return static_cast<size_t>(range_count(f, kMaxGemmCtas, nkv)) * nkv * 2 * tile_rows(f);
}

// A launch's schedule and pieces: [plan][places][begins][bases][pieces][o][(m, l)]
struct Part {
  size_t places, begins, bases, pieces, part_o, part_ml, total;
  Part(Form f, int nkv, size_t items, size_t prefix_items) {
    const size_t rows = piece_rows(f, nkv), ranges = range_count(f, kMaxGemmCtas, nkv);
    places = align_up(sizeof(Plan), kWsAlign);
    begins = places + align_up(ranges * sizeof(Place), kWsAlign);
    bases = begins + align_up((ranges + 1) * sizeof(int), kWsAlign);
    pieces = bases + align_up((items + 1) * sizeof(int2), kWsAlign);
    part_o = pieces + align_up((prefix_items + items) * sizeof(Pieces), kWsAlign);
    part_ml = part_o + align_up(rows * kHD * sizeof(float), kWsAlign);
    total = part_ml + align_up(rows * sizeof(float2), kWsAlign);
  }
  void fill(Args &a, char *p) const {
    a.plan = reinterpret_cast<Plan *>(p);
    a.places = reinterpret_cast<Place *>(p + places);
    a.begins = reinterpret_cast<int *>(p + begins);
    a.bases = reinterpret_cast<int2 *>(p + bases);
    a.pieces = reinterpret_cast<Pieces *>(p + pieces);
    a.part_o = reinterpret_cast<float *>(p + part_o);
    a.part_ml = reinterpret_cast<float2 *>(p + part_ml);
  }
};

size_t row_tiles(Form f, long long rows) { return static_cast<size_t>((rows + tile_rows(f) - 1) / tile_rows(f)); }

// With a prefix: one launch for both when the prefix's rows (all requests' rows) fit the
// kernels for few rows, else the prefix has a launch of its own.
bool prefix_apart(int B, long long rows) { return form_of(B * rows) == kShared && form_of(rows) != kShared; }

// At least the cost of a launch's schedule.
long long most_cost(const Args &a, int cache_len) {
  return static_cast<long long>(a.PRT) * (a.P / kTcKeys + 1 + kItemCost) +
         static_cast<long long>(a.B) * a.RT * (cache_len / kTcKeys + 2 + kItemCost);
}

}  // namespace

bool cache_map(CUtensorMap *map, const void *ptr, int B, int T, int nkv, int keys) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {kHD, static_cast<cuuint64_t>(nkv), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(B)};
  const cuuint64_t row = static_cast<cuuint64_t>(nkv) * kHD * 2;
  cuuint64_t strides[3] = {kHD * 2, row, row * static_cast<cuuint64_t>(T)};
  cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(keys), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool shape_ok(Kind kind, int B, int nr, int nq, int nkv, int cache_len, int prefix_len) {
  if (B > (1 << 16) || nq > 4096 || nkv > 1024 || cache_len > kMaxCacheLen || prefix_len > kMaxCacheLen ||
      static_cast<long long>(B) * nr > (1 << 20))
    return false;
  const long long rows = static_cast<long long>(nr) * (nq / nkv);
  if (kind == kScored && rows > kMaxScoredRows) return false;
  if (B * rows >= (1LL << 31)) return false;
  // the schedule counts units (row tiles x key tiles) in 32 bits
  auto units = [](long long n, Form f, long long r, long long keys) {
    return static_cast<double>(n) * ((r + tile_rows(f) - 1) / tile_rows(f)) * (keys / tile_keys(f) + 2);
  };
  const Form f = form_of(rows), pf = form_of(B * rows);
  return units(B, f, rows, cache_len) + units(1, pf, B * rows, prefix_len) < 2e9 &&
         units(B, pf, rows, cache_len) < 2e9;
}

// [header][requests' part][prefix's part][prefix or scored: rows' o, (m, l)][scored: row scores]
size_t workspace_bytes(Kind kind, int B, int nr, int nq, int nkv, int cache_len) {
  const size_t nrow = static_cast<size_t>(B) * nr * nq;
  const long long rows = static_cast<long long>(nr) * (nq / nkv);
  const Form f = form_of(rows);
  size_t part = Part(f, nkv, B * row_tiles(f, rows), 0).total, n = kWsAlign;
  if (kind == kPrefix) {   // (without a prefix the call takes the requests' form)
    const Form pf = form_of(B * rows);
    if (prefix_apart(B, rows))
      n += Part(kShared, nkv, 0, row_tiles(kShared, B * rows)).total;
    else
      part = std::max(part, Part(pf, nkv, B * row_tiles(pf, rows), row_tiles(pf, B * rows)).total);
    n += align_up(2 * nrow * kHD * sizeof(float), kWsAlign) + align_up(2 * nrow * sizeof(float2), kWsAlign);
  }
  n += part;
  if (kind == kScored) {
    n += Part(kShared, nkv, B * row_tiles(f, rows), 0).total + align_up(nrow * sizeof(float2), kWsAlign);
    const size_t s_ld = (static_cast<size_t>(cache_len) + 1) / 2 * 2;
    if (f == kMma) n += align_up(nrow * s_ld * sizeof(float), kWsAlign);
  }
  return n;
}

dspark_status_t launch(Kind kind, const Call &c, void *ws, cudaStream_t stream) {
  Args a = {};
  a.q = c.q;
  a.k_cache = c.k_cache;
  a.v_cache = c.v_cache;
  a.k_prefix = c.k_prefix;
  a.v_prefix = c.v_prefix;
  a.lens = c.lens;
  a.out = c.out;
  a.scores_in = c.scores_in;
  a.scores_out = c.scores_out;
  a.decay = c.decay;
  a.B = a.sB = c.B;
  a.nr = c.nr;
  a.nq = c.nq;
  a.nkv = c.nkv;
  a.grp = c.nq / c.nkv;
  a.cache_len = c.cache_len;
  a.P = c.prefix_len;
  a.window = c.window;
  a.sinks = c.sinks;
  a.causal = c.causal;
  a.rows = c.nr * a.grp;
  a.prows = c.prefix_len > 0 ? c.B * a.rows : 0;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(kHD)));
  const int sms = std::min(device_sm_count(), kMaxGemmCtas);
  if (sms <= 0) return DSPARK_ERR_NO_DEVICE;
  const bool apart = c.prefix_len > 0 && prefix_apart(c.B, a.rows);
  const Form f = apart ? form_of(a.rows) : form_of(std::max(a.rows, a.prows));
  const int rw = tile_rows(f);
  a.groups = range_count(f, sms, c.nkv);
  a.RT = static_cast<int>(row_tiles(f, a.rows));
  a.PRT = apart ? 0 : static_cast<int>(row_tiles(f, a.prows));
  // (the join by range, for more items than ranges, reads the plan; with a launch for the
  // prefix, thousands of joining warps would each work the schedule out: 14 us -> 18)
  a.direct = !apart && static_cast<long long>(c.B) * a.RT <= kDirectItems &&
             (c.prefix_len > 0 || c.B * a.RT <= a.groups) &&
             most_cost(a, c.cache_len) < (1LL << 32) / kMaxRanges;

  char *p = static_cast<char *>(ws);
  a.status = reinterpret_cast<int *>(p);
  p += kWsAlign;
  const Part part(f, c.nkv, c.B * row_tiles(f, a.rows), a.PRT);
  part.fill(a, p);
  p += part.total;
  Args pre = a;   // the prefix's own launch
  a.late_wait = apart ? 1 : 0;
  if (apart) {
    pre.sB = 0;
    pre.ordinary = 1;   // (the launch behind it does not wait: ragged.cuh, wait_first)
    pre.PRT = static_cast<int>(row_tiles(kShared, a.prows));
    const Part pp(kShared, c.nkv, 0, pre.PRT);
    pre.groups = range_count(kShared, sms, c.nkv);
    pp.fill(pre, p);
    p += pp.total;
  }
  const size_t nrow = static_cast<size_t>(c.B) * c.nr * c.nq;
  if (kind == kPrefix) {
    a.row_o = pre.row_o = reinterpret_cast<float *>(p);
    p += align_up(2 * nrow * kHD * sizeof(float), kWsAlign);
    a.row_ml = pre.row_ml = reinterpret_cast<float2 *>(p);
    const Args &src = apart ? pre : a;
    const Form sf = apart ? kShared : f;
    a.pre = {src.pieces, src.part_o, src.part_ml, tile_rows(sf), src.groups};
  }
  Args second = a;   // the scored form's second pass
  if (kind == kScored) {
    const Part sp(kShared, c.nkv, c.B * row_tiles(f, a.rows), 0);
    second.groups = range_count(kShared, sms, c.nkv);
    sp.fill(second, p);
    p += sp.total;
    a.row_ml = second.row_ml = reinterpret_cast<float2 *>(p);
    p += align_up(nrow * sizeof(float2), kWsAlign);
    a.smat = reinterpret_cast<float *>(p);
    a.s_ld = (c.cache_len + 1) / 2 * 2;
  }
  const bool weights = kind == kScored && f != kMma;
  dspark_status_t st = DSPARK_OK;
  if (!a.direct) st = plan_launch(a, f, apart ? &pre : weights ? &second : nullptr, kind, stream);
  if (st != DSPARK_OK) return st;
  if (apart && (st = tc_launch(pre, kShared, stream)) != DSPARK_OK) return st;
  st = f == kMma ? mma_launch(a, kind == kScored, stream) : tc_launch(a, f, stream);
  if (st != DSPARK_OK) return st;
  st = join_launch(a, rw, kind == kScored, stream);
  if (st != DSPARK_OK || kind != kScored) return st;
  return weights ? weights_launch(second, stream) : columns_launch(a, stream);
}

}  // namespace ragged
}  // namespace dspark
