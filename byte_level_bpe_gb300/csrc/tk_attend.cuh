// tk_attend.cuh -- what the attention kernels share: the requests, how the work is divided over
// the workers of a grid, and which keys a row sees.
#pragma once
#include "tk_blackwell.cuh"
#include "tk_kv.cuh"

namespace tk {

struct AttendArgs {
  const void* q;
  int64_t q_stride;
  int hq, hk, group;
  const int64_t* off;
  int64_t R, T, max_new;
  const int32_t* len;
  const int32_t* table;
  int64_t table_stride, table_width;
  const int64_t* mask;
  float scale_log2;
  void* out;
  float* lse;
  KvStatus* status;
  const void* v;
  int64_t n_blocks, s_block, s_head, s_token;
  int log2_bs;
  float* part;         // partial outputs, see the kernels
  unsigned* counters;  // [2 gridDim.x][2] of a divided unit, by its first worker: pieces that are done, joined
  int window, sinks;   // tilings with WIN: a token sees the `window` places up to its own, and the first `sinks`
  const float* k_scale;  // of a cache in 8 bits
  const float* v_scale;
  uint64_t per_group;  // 2^64 / group rounded up, 0 for a group of 1
};

// x / a.group, x from 0 on: 2^64 / group is off by less than 1, so x times it by less than 2^32.
__device__ __forceinline__ int by_group(const AttendArgs& a, int x) { return a.per_group ? (int)__umul64hi((uint64_t)x, a.per_group) : x; }

// A request as the schedule sees it.
struct Request {
  int t0;  // its first row of q
  int n, ctx, len;  // n < 0: the offsets decrease
  bool good;
};

__device__ __forceinline__ Request load_request(const AttendArgs& a, int64_t r) {
  Request q;
  const int64_t o = a.off[r], e = a.off[r + 1], len = a.len[r];
  // rows that cannot be taken are written as zeros: inside the output whatever the offsets say,
  // and, as long as these do not decrease, outside the other requests' rows
  const int64_t t0 = max((int64_t)0, min(o, a.T)), n = max((int64_t)0, min(e, a.T)) - t0;
  q.good = o >= 0 && e <= a.T && n >= 0 && n <= a.max_new && (!a.mask || n <= KV_TREE_MAX) && len >= n &&
           len <= a.table_width << a.log2_bs;
  q.t0 = (int)t0;
  q.n = (int)n;
  q.len = q.good ? (int)len : 0;
  q.ctx = q.good ? (int)(len - n) : 0;
  return q;
}

// How a kernel cuts its work.  A unit is ROWS query rows (tokens x query heads of one key head) of a
// request; its keys are read in steps of STEP neighbouring keys, and STEPS of them are a tile.  WIN: the
// call has a window.  The others are costs in tiles, see the kernels.
template <int ROWS_, int STEP_, int STEPS_, bool WIN_, int UNIT_COST_, int MIN_SHARE_, int SNAP_, int PADDED_MORE_, bool QUARTER_>
struct Tiling {
  static constexpr int ROWS = ROWS_, STEP = STEP_, STEPS = STEPS_;
  static constexpr bool WIN = WIN_;
  static constexpr int UNIT_COST = UNIT_COST_, MIN_SHARE = MIN_SHARE_, SNAP = SNAP_;
  // what a worker may do more if it has a single piece for that, in tiles, and a quarter
  static constexpr int PADDED_MORE = PADDED_MORE_;
  static constexpr bool QUARTER = QUARTER_;
  static_assert(SNAP >= UNIT_COST && MIN_SHARE >= 2 * SNAP, "a piece has at least one tile");
};

// The keys that a unit reads: those before `keys`, but for `skip` steps from step `head` on
// (between the first places and the window of the unit's first token).
struct Span {
  int keys, head, skip;
};
template <class S>
__device__ __forceinline__ Span unit_span(const AttendArgs& a, const Request& q, int row0) {
  Span x = {q.len, 0, 0};
  if (!q.good) return x;
  if (!a.mask) x.keys = q.ctx + by_group(a, min(q.n * a.group, row0 + S::ROWS) - 1) + 1;
  if (S::WIN) {
    const int low = q.ctx + (a.mask ? 0 : by_group(a, row0)) + 1 - a.window;
    x.head = (a.sinks + S::STEP - 1) / S::STEP;
    x.skip = max(0, low / S::STEP - x.head);
  }
  return x;
}
template <class S>
__device__ __forceinline__ int span_steps(const Span& x) {
  return (x.keys + S::STEP - 1) / S::STEP - (S::WIN ? x.skip : 0);
}
// Tiles of a unit: at least one, which writes the rows.
template <class S>
__device__ __forceinline__ int span_tiles(const Span& x) {
  return max(1, (span_steps<S>(x) + S::STEPS - 1) / S::STEPS);
}

// How the work is divided.  It is one line of units (request, row tile, key
// head), each UNIT_COST + its tiles long; worker w has it from w * share to
// (w + 1) * share.  Long caches are so divided over workers and short ones
// gathered in one; a cut within SNAP of a unit's start or end moves there.
// Padded: there are fewer units than workers; a unit's length is rounded up to
// whole shares and divided evenly over its workers, each of which has that one piece.
// (A line of 2^31 and more is refused; from 2^30 on one may be: a request counts as up to 1,024 more.)
struct Plan {
  int share;
  bool padded;
};

struct UnitSum {
  int length, units, longest;
};
// shared: a whole warp has the request, each lane some of its row tiles, and all get the sum.
template <class S>
__device__ __forceinline__ UnitSum request_work(const AttendArgs& a, const Request& q, const Plan& plan, bool shared) {
  UnitSum w = {0, 0, 0};
  int64_t length = 0;
  const int rows = q.n * a.group;
  const bool same = a.mask || !q.good || rows <= S::ROWS;  // every row tile has the request's keys
  shared = shared && !same;
  const int step = shared ? 32 * S::ROWS : S::ROWS;
#pragma unroll 1
  for (int64_t row0 = shared ? threadIdx.x % 32 * S::ROWS : 0; row0 < rows; row0 += step) {
    const int cost = span_tiles<S>(unit_span<S>(a, q, (int)row0)) + S::UNIT_COST;
    const int tiles = same ? (rows + S::ROWS - 1) / S::ROWS : 1;
    length += (int64_t)(plan.padded ? ((unsigned)(cost + plan.share - 1) / (unsigned)plan.share) * plan.share : cost) * tiles;
    w.units += tiles;
    w.longest = max(w.longest, cost);
    if (same) break;
  }
  if (shared) {
#pragma unroll 1
    for (int o = 1; o < 32; o *= 2) {
      length += __shfl_xor_sync(0xffffffffu, length, o);
      w.units += __shfl_xor_sync(0xffffffffu, w.units, o);
      w.longest = max(w.longest, __shfl_xor_sync(0xffffffffu, w.longest, o));
    }
  }
  w.length = (int)min(length * a.hk, (int64_t)INT32_MAX);
  w.units *= a.hk;
  return w;
}

struct Piece {
  int t0, r, h;       // first row of q, request, key head
  int row0, rows;     // rows of the unit among the request's tokens x group
  int n, ctx, len;    // of the request; ctx = len = 0 if it cannot be taken
  int open;           // keys that every row of the unit sees, but those from sinks to `shut`
  int shut;           // with a window
  int keys, lo, hi;   // keys of the unit; tiles of this piece
  int head, skip;     // of its span
  int first, pieces;  // the worker with the unit's tile 0; workers it is divided over
  int valid;          // 0 = no more, 1 = a request that cannot be taken
};
template <class S>
struct Walk {
  Plan plan;
  int from, to;  // the worker's part of the line
  int u, r;      // where the next unit starts, and its request
  Request q;
  int row0, h;                         // the unit's row tile and head
  Span span;                           // of the row tile's units
  int cost, pieces, size, length;      // theirs; padded: what they are divided into
  bool loaded;

  __device__ __forceinline__ void row_tile(const AttendArgs& a) {
    span = unit_span<S>(a, q, row0);
    cost = length = span_tiles<S>(span) + S::UNIT_COST;
    if (plan.padded) {
      pieces = (unsigned)(cost + plan.share - 1) / (unsigned)plan.share;
      size = (unsigned)(cost + pieces - 1) / (unsigned)pieces;
      length = pieces * plan.share;
    }
  }
  // A whole warp, before its first piece: on to the row tile of the first request in which the worker's part
  // begins, 32 of them at a time (a prompt of 2,000 tokens has 63, one after the other they took 10 us).
  __device__ __forceinline__ void seek(const AttendArgs& a) {
    if (u >= to || r >= a.R) return;
    q = load_request(a, r);
    const int lane = threadIdx.x & 31, rows = q.n * a.group;
    if (rows <= S::ROWS) return;
    loaded = true;
    row0 = h = 0;
    for (int64_t first = 0; first < rows; first += 32 * S::ROWS) {
      const int64_t mine = first + lane * S::ROWS;
      int all = 0;
      if (mine < rows) {
        row0 = (int)mine;
        row_tile(a);
        all = length * a.hk;
      }
#pragma unroll 1
      for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += x;
      }
      const uint32_t there = __ballot_sync(0xffffffffu, mine < rows && u + all > from);
      const int at = there ? __ffs(there) - 1 : 31;
      const int passed = __shfl_sync(0xffffffffu, all, there ? max(at - 1, 0) : 31);
      if (!there || at > 0) u += passed;
      row0 = (int)min(first + at * S::ROWS, (int64_t)INT32_MAX);
      if (there) break;
    }
    if (row0 < rows) {
      row_tile(a);
    } else {  // never: the request holds what the worker begins with
      r++;
      loaded = false;
    }
  }
  __device__ __forceinline__ bool next(const AttendArgs& a, Piece& x) {
    for (;;) {
      if (u >= to || r >= a.R) break;
      if (!loaded) {
        q = load_request(a, r);
        if (q.n <= 0) {
          r++;
          continue;
        }
        row0 = h = 0;
        loaded = true;
        row_tile(a);
      }
      if (u + length <= from) {  // heads before this worker
        const int skip = min(a.hk - h, (int)((unsigned)(from - u) / (unsigned)length));
        u += skip * length;
        h += skip;
      }
      if (h == a.hk) {
        h = 0;
        row0 += S::ROWS;
        loaded = row0 < q.n * a.group;
        if (loaded) row_tile(a);
        else r++;
        continue;
      }
      const int lo = cut(from - u), hi = cut(to - u), at = u;
      u += length;
      h++;
      if (hi <= lo) continue;
      x.t0 = q.t0;
      x.r = r;
      x.h = h - 1;
      x.row0 = row0;
      x.rows = min(S::ROWS, q.n * a.group - row0);
      x.n = q.n;
      x.ctx = q.ctx;
      x.len = q.len;
      x.open = !q.good ? 0 : a.mask ? q.ctx : q.ctx + by_group(a, row0) + 1;
      if (S::WIN) {
        x.shut = q.ctx + (a.mask ? min(q.n, KV_TREE_MAX) : by_group(a, row0 + x.rows - 1) + 1) - a.window;
        x.head = span.head;
        x.skip = span.skip;
      }
      x.keys = span.keys;
      x.lo = max(0, lo - S::UNIT_COST);
      x.hi = hi - S::UNIT_COST;
      x.first = 0;
      x.pieces = 1;
      if (lo > 0 || hi < cost) {
        x.first = (unsigned)(at + (plan.padded ? 0 : S::SNAP)) / (unsigned)plan.share;
        x.pieces = plan.padded ? pieces : (int)((unsigned)(at + cost - S::SNAP - 1) / (unsigned)plan.share) - x.first + 1;
      }
      x.valid = 1 + q.good;
      return true;
    }
    x.valid = 0;
    return false;
  }
  // a worker's end `in` after the unit's start, as a cut of the unit
  __device__ __forceinline__ int cut(int in) const {
    if (in <= 0) return 0;
    if (in >= length) return cost;
    if (plan.padded) return min(cost, (int)((unsigned)in / (unsigned)plan.share) * size);
    return in <= S::SNAP ? 0 : in >= cost - S::SNAP ? cost : in;
  }
};

// Rows of no request are zeros, so that padding carries nothing on.  Rarely run: in line it cost
// 64 drafted tokens over 131k 1% (204 instead of 202 us).
template <int D>
__device__ __noinline__ void zero_rows(void* out, float* lse, int hq, int64_t from, int64_t to) {
  const int64_t me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, all = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = from * hq * (D / 8) + me; i < to * hq * (D / 8); i += all) static_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
  if (lse)
    for (int64_t i = from * hq + me; i < to * hq; i += all) lse[i] = -INFINITY;
}

// The plan, and where the CTA's workers start on its line: the requests' lengths added up, each
// thread a run of them.  s_sum: 4 * THREADS / 32 words; s_walk: of each of the CTA's workers its first
// request, and where that starts.  The caller synchronises after it.  Returns the line's length.
template <class S, int THREADS, int WORKERS, int D>
__device__ __forceinline__ int make_plan(const AttendArgs& a, Plan& plan, int* s_sum, int* s_walk) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* s_units = s_sum + THREADS / 32;
  int* s_longest = s_units + THREADS / 32;
  int* s_coarse = s_longest + THREADS / 32;
  plan = {1, false};
  int total;
  // few requests are a warp's each, which counts their row tiles together; of many a thread has a run
  const int R = (int)a.R;
  const bool few = R <= THREADS / 32;
  const int per = (R + THREADS - 1) / THREADS;
  const int r0 = few ? min(R, warp) : min(R, tid * per), r1 = few ? min(R, warp + 1) : min(R, r0 + per);
  const bool counts = !few || lane == 0;
  int mine = 0, units = 0, longest = 0, before, coarse = 0;
  const int64_t head = R ? a.off[0] : 0, tail = R ? a.off[R] : 0;
  for (int r = r0; r < r1; r++) {
    const Request q = load_request(a, r);
    if (q.n < 0) {  // requests over each other: any amount of work, and of rows with two answers
      coarse = 1 << 21;
      break;
    }
    if (!q.good && blockIdx.x == 0 && counts && atomicCAS(&a.status->code, 0, TK_E_LIMIT) == 0) a.status->request = r;
    const UnitSum w = request_work<S>(a, q, plan, few);
    if (!counts) break;
    mine += w.length;
    units += w.units;
    longest = max(longest, w.longest);
    coarse = min(coarse + (w.length >> 10) + 1, 1 << 21);
  }
  // the sum over the threads before this one, and over all
  auto scan = [&](int x, int& all) {
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int b = incl - x;
    all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; w++) {
      const int y = s_sum[w];
      if (w < warp) b += y;
      all += y;
    }
    return b;
  };
  units = __reduce_add_sync(0xffffffffu, units);
  longest = __reduce_max_sync(0xffffffffu, longest);
  coarse = __reduce_add_sync(0xffffffffu, coarse);
  if (lane == 0) {
    s_units[warp] = units;
    s_longest[warp] = longest;
    s_coarse[warp] = coarse;
  }
  before = scan(mine, total);
  units = coarse = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; w++) {
    units += s_units[w];
    longest = max(longest, s_longest[w]);
    coarse += s_coarse[w];
  }
  // more than the line's 32 bits hold, or offsets that decrease: nothing is done then
  const bool much = coarse >= 1 << 21;
  if (much) {
    if (blockIdx.x == 0 && tid == 0 && atomicCAS(&a.status->code, 0, TK_E_LIMIT) == 0) a.status->request = -1;
    total = mine = units = 0;
  }
  // rows of no request are zeros, so that padding carries nothing on; after the last and before the first
  if (much) {
    zero_rows<D>(a.out, a.lse, a.hq, 0, a.T);
  } else if (head > 0 || tail < a.T) {
    zero_rows<D>(a.out, a.lse, a.hq, 0, min(head, a.T));
    zero_rows<D>(a.out, a.lse, a.hq, max(tail, (int64_t)0), a.T);
  }
  const int workers = gridDim.x * WORKERS;
  auto over = [](int x, int y) { return (int)((unsigned)(x + y - 1) / (unsigned)y); };
  plan.share = max(S::MIN_SHARE, over(total, workers));
  // (a padded line is at most a quarter longer and 8 * workers: it fits 31 bits with what it is below here)
  if (units > 0 && units < workers && total <= 1 << 30) {
    // shares that give the units no more workers than there are
    const int share = max(S::MIN_SHARE, min(over(longest, workers / units), over(total, workers - units)));
    // What a worker may do more if it has a single piece for that.  Up to 128 rows memory is the
    // bound, which fewer workers reach too, so that may be a quarter: 32 trees of 16 over 8k, 256
    // units for 304 workers, take 159 us padded (128 tiles each) and 189 us divided evenly (108),
    // 30 trees of 8 over 3k 62 and 77, one token of 32 requests over 8k of head_dim 64 109 and 106.  The 8 tiles
    // are for more rows: two trees of 64 over 30k take 67 us padded and 82 us not.
    if (share <= plan.share + S::PADDED_MORE + (S::QUARTER ? plan.share / 4 : 0)) {
      plan.share = share;
      plan.padded = true;
      mine = 0;
      for (int r = r0; r < r1; r++) {
        const int c = request_work<S>(a, load_request(a, r), plan, few).length;
        if (counts) mine += c;
      }
      __syncthreads();  // s_sum has been read
      before = scan(mine, total);
    }
  }
  for (int w = 0; w < WORKERS; w++) {
    const int x = (blockIdx.x * WORKERS + w) * plan.share;
    if (x < before || x >= before + mine) continue;
    int r = r0, at = before;
    for (; r < r1 - 1; r++) {
      const int c = request_work<S>(a, load_request(a, r), plan, false).length;  // (of few requests r0 is the last)
      if (x < at + c) break;
      at += c;
    }
    s_walk[2 * w] = r;
    s_walk[2 * w + 1] = at;
  }
  return total;
}

// Keys that a row sees, 32 from `first` on as bits, or one of them.
template <bool WIN>
struct Seen {
  int ctx, last;   // chain: keys up to `last`
  uint64_t mask;   // tree: drafted tokens
  bool tree;
  int low, sinks;  // WIN: of the context (a chain's new tokens too) those from `low` on and the first `sinks`

  // piece x, row gr of its request's
  __device__ __forceinline__ void set(const AttendArgs& a, const Piece& x, bool live, int tok) {
    tree = a.mask != nullptr;
    ctx = x.ctx;
    last = x.valid == 2 ? x.ctx + tok : -1;
    mask = 0;
    int at = x.ctx + tok;
    if (tree && live && x.valid == 2) {
      mask = (uint64_t)a.mask[x.t0 + tok];
      if (x.n < 64) mask &= (1ull << x.n) - 1;
      at = x.ctx + __popcll(mask & ~(1ull << tok));
    }
    low = WIN ? max(0, at + 1 - a.window) : 0;
    sinks = WIN ? a.sinks : 0;
  }
  static __device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }
  __device__ __forceinline__ uint32_t bits(int first) const {
    uint32_t far = 0;  // places outside the window
    if (WIN) far = below(low - first) & ~below(sinks - first);
    if (!tree) return below(last + 1 - first) & ~far;
    const int sh = first - ctx;
    if (sh <= -32) return ~far;
    if (sh >= 64) return 0u;
    return sh >= 0 ? (uint32_t)(mask >> sh) : ((uint32_t)mask << -sh) | (((1u << -sh) - 1) & ~far);
  }
  __device__ __forceinline__ bool has(int j) const {
    if (WIN && j < low && j >= sinks && (!tree || j < ctx)) return false;
    return tree ? j < ctx || (j - ctx < 64 && ((mask >> (j - ctx)) & 1)) : j <= last;
  }
};

// Over 8 bits, see tk_attend8.cu: the bounds M and R of a row that has seen nothing, the exponent of a weight at R, log2 of a
// scale of 0; log2 of a values' scale, finite whatever is in a place that nobody sees; and d.
constexpr float E8_MOST = 3.402823466e38f, E8_TOP = 15.f, E8_NONE = -1000.f;
__device__ __forceinline__ float e8_log2(float vs) { return fmaxf(fminf(log2f(vs), 128.f), E8_NONE); }
__device__ __forceinline__ float e8_shift(float lv, float M, float R) { return fmaxf(lv + (M - R + E8_TOP), -60.f); }

template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const typename Pair<T>::type p = Pair<T>::down(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The kernels' launches; rows: of a request and key head, at most.  With a window over a cache in 16 bits
// (tk_attend_window.cu), over a cache in 8 bits (tk_attend8.cu, of few rows), and of many rows (tk_attend8_mma.cu).
cudaError_t attend_windowed(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st);
cudaError_t attend8(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st);
cudaError_t attend8_many(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st);

}  // namespace tk
