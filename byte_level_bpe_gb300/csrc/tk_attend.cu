// tk_attend.cu -- attention of new and drafted tokens over the paged cache
// (tk_kv_attend): o = sum_j softmax_j(scale q.k_j) v_j over the keys j that a
// token sees.
//
// The query rows of one request and key head (tokens x query heads of that key
// head) are the rows of the products S = Q K^T and O = P V on the 5th-generation
// tensor cores; 128 rows are one tile whether they are all in use or not: for 128
// keys the two products take about 1,300 cycles against the 2,850 that their
// 64 KB of keys and values take from HBM (head_dim 128), so padding costs nothing while
// memory is the bound.  With a running maximum m and sum l,
//   p_j = 2^(c (s_j - m) + UP), c = scale log2(e),  l += sum p_j,  O += P V,
// and O is rescaled in tensor memory only when m grows by more than 2^8 in p
// (p and l are relative to the same m and UP, so the quotient is exact either way).
// S, m, l and O are fp32; P is rounded to the cache's type, which the tensor
// cores ask for, and l sums what was rounded: an error of half an ulp in each weight, but
// none in a weight that is nearly alone (summed before the rounding, the result's error
// against 64 bits came to 1.6 times that of rounding it alone; so it is 1.1 to 1.4 times, for
// 4% of the time of the second case below).
//
// Bounds, on one GB300: HBM up to 128 rows (one token of 128 requests over 6k,
// 3.25 GB: 488 us, 6.7 TB/s); above, the tensor cores and the latency of the chain from one
// tile's scores to the next one's (64 drafted tokens over 131k, 512 rows a head: 219 us,
// 1.25 PFLOP/s; 202 with the keys in L2 from the call before); a short call its chain of
// first accesses (200 keys: 12 us).
#include <algorithm>
#include <new>
#include <type_traits>

#include "tk_blackwell.cuh"
#include "tk_kv.cuh"

namespace tk {

constexpr int AT_THREADS = 384;  // loads and products of two streams (4 warps), their softmax (2 x 4 warps)
// How the work is divided, in tiles.  Times of one call in a replayed graph, in us.
// What starting a unit costs: with 1, six prompts of 2,000 tokens take 484 instead of 365 and
// one token of 32 requests over 3k (head_dim 64) 53 instead of 45; with 6, one token of 128
// requests over 6k 490 instead of 481, the prompts 359.
constexpr int AT_UNIT_COST = 3;
// Least share of a worker: with 6 (and a snap of 3) one token over 200 takes 13.3 instead of 11.8;
// with 16 one token of 8 requests over 2k 24.6 instead of 23.0.
constexpr int AT_MIN_SHARE = 8;
// A unit is not cut nearer to its ends than this: with 3, 24 trees of 9 over 1.5k (head_dim 64)
// take 41.8 instead of 41.3; with 6 (and a least share of 12) 38.6, the others the same.
constexpr int AT_SNAP = 4;
static_assert(AT_SNAP >= AT_UNIT_COST && AT_MIN_SHARE >= 2 * AT_SNAP, "a piece has at least one tile");

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
  float* part;         // partial outputs, see part_at
  unsigned* counters;  // [2 gridDim.x][2] of a divided unit, by its first stream: pieces that are done, joined
};

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

// Keys that the rows [row0, row0 + ROWS) of a request read, and their tiles (at
// least one: it writes the rows).
template <int ROWS>
__device__ __forceinline__ int unit_keys(const AttendArgs& a, const Request& q, int row0) {
  if (a.mask || !q.good) return q.len;
  return q.ctx + (min(q.n * a.group, row0 + ROWS) - 1) / a.group + 1;
}
// Tiles of a 256-row unit have 128 keys, the others' 64 (see AttendShape).
template <int ROWS>
__device__ __forceinline__ int key_tiles(int keys) {
  constexpr int KEYS = ROWS == 256 ? 128 : 64;
  return max(1, (keys + KEYS - 1) / KEYS);
}

// How the work is divided.  It is one line of units (request, row tile, key
// head), each AT_UNIT_COST + its key tiles long; worker w has it from w * share to
// (w + 1) * share.  Long caches are so divided over workers and short ones
// gathered in one; a cut within AT_SNAP of a unit's start or end moves there.
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
template <int ROWS>
__device__ __forceinline__ UnitSum request_work(const AttendArgs& a, const Request& q, const Plan& plan) {
  UnitSum w = {0, 0, 0};
  int64_t length = 0;
  const int rows = q.n * a.group;
  const bool same = a.mask || !q.good || rows <= ROWS;  // every row tile has the request's keys
  for (int row0 = 0; row0 < rows; row0 += ROWS) {
    const int cost = key_tiles<ROWS>(unit_keys<ROWS>(a, q, row0)) + AT_UNIT_COST;
    const int tiles = same ? (rows + ROWS - 1) / ROWS : 1;
    length += (int64_t)(plan.padded ? ((unsigned)(cost + plan.share - 1) / (unsigned)plan.share) * plan.share : cost) * tiles;
    w.units += tiles;
    w.longest = max(w.longest, cost);
    if (same) break;
  }
  w.length = (int)min(length * a.hk, (int64_t)INT32_MAX);
  w.units *= a.hk;
  return w;
}

struct Piece {
  int t0, r, h;       // first row of q, request, key head
  int row0, rows;     // rows of the unit among the request's tokens x group
  int n, ctx, len;    // of the request; ctx = len = 0 if it cannot be taken
  int open;           // keys that every row of the unit sees
  int keys, lo, hi;   // keys of the unit; tiles of this piece
  int first, pieces;  // the worker with the unit's tile 0; workers it is divided over
  int valid;          // 0 = no more, 1 = a request that cannot be taken
};
constexpr int AT_PIECES = 4;  // handed over ahead

template <int ROWS>
struct Walk {
  Plan plan;
  int from, to;  // the worker's part of the line
  int u, r;      // where the next unit starts, and its request
  Request q;
  int row0, h;                         // the unit's row tile and head
  int keys, cost, pieces, size, length;  // of the row tile's units; padded: what they are divided into
  bool loaded;

  __device__ __forceinline__ void row_tile(const AttendArgs& a) {
    keys = unit_keys<ROWS>(a, q, row0);
    cost = length = key_tiles<ROWS>(keys) + AT_UNIT_COST;
    if (plan.padded) {
      pieces = (unsigned)(cost + plan.share - 1) / (unsigned)plan.share;
      size = (unsigned)(cost + pieces - 1) / (unsigned)pieces;
      length = pieces * plan.share;
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
        row0 += ROWS;
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
      x.rows = min(ROWS, q.n * a.group - row0);
      x.n = q.n;
      x.ctx = q.ctx;
      x.len = q.len;
      x.open = !q.good ? 0 : a.mask ? q.ctx : q.ctx + row0 / a.group + 1;
      x.keys = keys;
      x.lo = max(0, lo - AT_UNIT_COST);
      x.hi = hi - AT_UNIT_COST;
      x.first = 0;
      x.pieces = 1;
      if (lo > 0 || hi < cost) {
        x.first = (unsigned)(at + (plan.padded ? 0 : AT_SNAP)) / (unsigned)plan.share;
        x.pieces = plan.padded ? pieces : (int)((unsigned)(at + cost - AT_SNAP - 1) / (unsigned)plan.share) - x.first + 1;
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
    return in <= AT_SNAP ? 0 : in >= cost - AT_SNAP ? cost : in;
  }
};

// The keys of a row among 32 from `first` on, as bits.
struct Seen {
  int ctx, last;     // chain: keys up to `last`
  uint64_t mask;     // tree: drafted tokens
  bool tree;
  __device__ __forceinline__ uint32_t bits(int first) const {
    if (!tree) {
      const int n = last + 1 - first;
      return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1;
    }
    const int sh = first - ctx;
    if (sh <= -32) return 0xffffffffu;
    if (sh >= 64) return 0u;
    return sh >= 0 ? (uint32_t)(mask >> sh) : ((uint32_t)mask << -sh) | ((1u << -sh) - 1);
  }
  __device__ __forceinline__ bool has(int j) const {
    return tree ? j < ctx || (j - ctx < 64 && ((mask >> (j - ctx)) & 1)) : j <= last;
  }
};

template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const typename Pair<T>::type p = Pair<T>::down(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// 16-bit halves with all exponent bits set (infinities and NaN): 0x8000 each.
template <class T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w);
template <>
__device__ __forceinline__ uint32_t nonfinite2<__nv_bfloat16>(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
template <>
__device__ __forceinline__ uint32_t nonfinite2<__half>(uint32_t w) {
  return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

// MODE 0 and 1: a CTA's two streams are workers of their own, with units of at
// most 32 or 128 rows (0: less room for queries, more for tiles in flight), so
// that one's starts and ends run under the other's tiles.  MODE 2: a CTA is one worker with
// units of 256 rows, each stream has 128 of them and both read every tile.  A stream
// has 128 columns of tensor memory for scores.  64-key tiles leave room for the
// scores of two, so that products run under the softmax of their own stream; with
// 128-key tiles they run under the other stream's, and read the queries half as often
// from shared memory (for 128 rows and 64 keys that is the products' bound: 48 cycles instead of 32 for
// k = 16).  64 drafted tokens over 131k take 218 us with the former and 204 with the latter (both
// before the sums of rounded weights).
template <int D, int MODE>
struct AttendShape {
  static constexpr int RINGS = MODE == 2 ? 1 : 2, ROWS = MODE == 0 ? 32 : MODE == 1 ? 128 : 256;
  static constexpr int Q_ROWS = MODE == 0 ? 32 : 128;  // of a stream
  static constexpr int KEYS = MODE == 2 ? 128 : 64, BUFS = 128 / KEYS;  // keys of a tile; tiles' scores in tensor memory
  static constexpr int Q = Q_ROWS * D * 2, STAGE = KEYS * D * 2;
  static constexpr int STAGES = (RINGS == 1 ? 160 : MODE == 0 ? 96 : 80) * 1024 / STAGE;  // of a ring
  static constexpr int RING = 2 * Q;
  // barriers: full and empty of the stages; pieces handed over and taken; per stream q, s (2), p (2), v, o ready, o free, drain,
  // turn
  static constexpr int BARS = RING + RINGS * STAGES * STAGE;
  static constexpr int N_BARS = RINGS * (2 * STAGES + 2 * AT_PIECES) + 2 * 10;
  static constexpr int PIECES = BARS + 8 * N_BARS;
  static constexpr int SMALL = PIECES + RINGS * AT_PIECES * (int)sizeof(Piece);
  // start of the walk (2 x 2), sums, units and longest of the warps, tensor memory, abort, non-finite values (2 x 8)
  static constexpr int TOTAL = SMALL + 16 + 16 * (AT_THREADS / 32) + 72;
  static_assert(SMALL % 8 == 0 && TOTAL <= 227 * 1024, "shared memory of one CTA");
};

// Partial output of a piece: [D / 4][128 rows][4] normalised, then [128] log2 of
// the row's sum (of rounded weights) and [128] what the sum before rounding is of it: lanes
// are rows, and neighbours in memory.  A stream has at most two: slot 1
// if it holds the unit's first tile.
template <int D>
__device__ __forceinline__ float* part_at(float* part, int stream, int slot) {
  return part + (int64_t)(stream * 2 + slot) * (128 * (D + 2));
}

// Warps 0 and 3 load (one per ring), warps 1 and 2 issue the products of streams
// 0 and 1, warps 4-7 and 8-11 are their softmax, a thread per row (two threads per row
// were slower: 267 instead of 222 us for 64 drafted tokens over 131k).  Tensor memory of a
// stream: scores (128 columns, the weights over the first half of a tile's) and O
// (128), 256 columns from 256 * stream.
// LSE: the log of the sum is wanted too, and summed before the rounding (64 drafted tokens over
// 131k, replayed: 204 us without it, 221 with it; up to 128 rows the softmax is not the bound, and it is always there).
// Rows of no request are zeros, so that padding carries nothing on.  Rarely run: in line it cost
// 64 drafted tokens over 131k 1% (204 instead of 202 us).
template <int D>
__device__ __noinline__ void zero_rows(void* out, float* lse, int hq, int64_t from, int64_t to) {
  const int64_t me = (int64_t)blockIdx.x * AT_THREADS + threadIdx.x, all = (int64_t)gridDim.x * AT_THREADS;
  for (int64_t i = from * hq * (D / 8) + me; i < to * hq * (D / 8); i += all) static_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
  if (lse)
    for (int64_t i = from * hq + me; i < to * hq; i += all) lse[i] = -INFINITY;
}

template <class T, int D, int MODE, bool LSE>
__global__ void __launch_bounds__(AT_THREADS, 1)
k_kv_attend(const AttendArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using L = AttendShape<D, MODE>;
  constexpr int ROWS = L::ROWS, KEYS = L::KEYS, BUFS = L::BUFS, HALVES = D / 64, NST = L::STAGES;
  constexpr bool BF = Pair<T>::BF;
  // fp16 weights have their range below 2^15: with m's weight at 2^7 those 2^8 above it (before O is
  // rescaled) still fit, and one is lost at 2^-32 of m's instead of 2^-25: a million keys that
  // are each just below come to half an ulp of one of m's weight.
  constexpr float UP = BF ? 0.f : 7.f;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle goes by address bits
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stream = warp < 4 ? (warp >> 1) : (warp - 4) >> 2;  // warps 0, 1 | 2, 3
  const int ring = MODE == 2 ? 0 : stream;
  const uint32_t s_ring = base + L::RING + ring * (NST * L::STAGE), s_q = base + stream * L::Q;
  const uint32_t b_full = base + L::BARS + ring * 8 * (2 * NST + 2 * AT_PIECES), b_empty = b_full + 8 * NST,
                 b_piece = b_empty + 8 * NST, b_taken = b_piece + 8 * AT_PIECES;
  const uint32_t b_q = base + L::BARS + L::RINGS * 8 * (2 * NST + 2 * AT_PIECES) + stream * 80, b_s = b_q + 8, b_p = b_s + 16,
                 b_v = b_p + 16, b_o = b_v + 8, b_free = b_o + 8, b_drain = b_free + 8, b_turn = b_drain + 8;
  Piece* s_piece = reinterpret_cast<Piece*>(smem + L::PIECES) + ring * AT_PIECES;
  int* s_walk = reinterpret_cast<int*>(smem + L::SMALL);  // of each worker: first request, where it starts
  int* s_sum = s_walk + 4;
  int* s_units = s_sum + AT_THREADS / 32;
  int* s_longest = s_units + AT_THREADS / 32;
  int* s_coarse = s_longest + AT_THREADS / 32;
  volatile int* s_int = reinterpret_cast<volatile int*>(s_coarse + AT_THREADS / 32);
  volatile int* abort = s_int + 1;
  volatile int* s_bad = s_int + 2 + 8 * ring;  // by piece

  if (base & 1023) {  // never: the swizzle would not hold
    if (tid == 0) a.status->code = TK_E_CUDA;
    return;
  }
  if (warp == 2) {
    for (int i = lane; i < L::N_BARS; i += 32) {
      int count = 1;
      const int in = i % (2 * NST + 2 * AT_PIECES), st = i - L::RINGS * (2 * NST + 2 * AT_PIECES);
      if (st < 0) {
        if (in >= NST && in < 2 * NST) count = MODE == 2 ? 2 : 1;                // empty: the streams that read the stage
        else if (in >= 2 * NST + AT_PIECES) count = MODE == 2 ? 10 : 5;          // taken: products and softmax warps
      } else {
        const int k = st % 10;
        count = k == 0 ? 128 : k == 3 || k == 4 || k == 7 ? 4 : 1;               // q, p, p, o free
      }
      bar_init(base + L::BARS + 8 * i, count);
    }
    fence_bar_init();
  }
  if (tid < 17) s_int[1 + tid] = 0;
  if (tid == 0 || tid == 96) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k));
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v));
  }
  if (warp == 1) tmem_alloc(smem_addr(const_cast<int*>(s_int)));

  // the block table on its way to L2, for the loads that follow the plan
  {
    const int64_t at = ((int64_t)blockIdx.x * AT_THREADS + tid) * 32;
    if (at < (a.R - 1) * a.table_stride + a.table_width) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table + at));
  }
  // the plan, and where the workers start on its line: the requests' lengths added up, each
  // thread a run of them
  constexpr int WORKERS = MODE == 2 ? 1 : 2;  // of a CTA
  Plan plan = {1, false};
  int total;
  {
    const int R = (int)a.R, per = (R + AT_THREADS - 1) / AT_THREADS;
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    int mine = 0, units = 0, longest = 0, before, coarse = 0;
    const int64_t head = R ? a.off[0] : 0, tail = R ? a.off[R] : 0;
    for (int r = r0; r < r1; r++) {
      const Request q = load_request(a, r);
      if (q.n < 0) {  // requests over each other: any amount of work, and of rows with two answers
        coarse = 1 << 21;
        break;
      }
      if (!q.good && blockIdx.x == 0 && atomicCAS(&a.status->code, 0, TK_E_LIMIT) == 0) a.status->request = r;
      const UnitSum w = request_work<ROWS>(a, q, plan);
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
      for (int w = 0; w < AT_THREADS / 32; w++) {
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
    for (int w = 0; w < AT_THREADS / 32; w++) {
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
    plan.share = max(AT_MIN_SHARE, over(total, workers));
    // (a padded line is at most a quarter longer and 8 * workers: it fits 31 bits with what it is below here)
    if (units > 0 && units < workers && total <= 1 << 30) {
      // shares that give the units no more workers than there are
      const int share = max(AT_MIN_SHARE, min(over(longest, workers / units), over(total, workers - units)));
      // What a worker may do more if it has a single piece for that.  Up to 128 rows memory is the
      // bound, which fewer workers reach too, so that may be a quarter: 32 trees of 16 over 8k, 256
      // units for 304 workers, take 159 us padded (128 tiles each) and 189 us divided evenly (108),
      // 30 trees of 8 over 3k 62 and 77, one token of 32 requests over 8k of head_dim 64 109 and 106.  The 8 tiles
      // are for more rows: two trees of 64 over 30k take 67 us padded and 82 us not.
      if (share <= plan.share + 8 + (MODE == 2 ? 0 : plan.share / 4)) {
        plan.share = share;
        plan.padded = true;
        mine = 0;
        for (int r = r0; r < r1; r++) mine += request_work<ROWS>(a, load_request(a, r), plan).length;
        __syncthreads();  // s_sum has been read
        before = scan(mine, total);
      }
    }
    for (int w = 0; w < WORKERS; w++) {
      const int x = (blockIdx.x * WORKERS + w) * plan.share;
      if (x < before || x >= before + mine) continue;
      int r = r0, at = before;
      for (; r < r1 - 1; r++) {
        const int c = request_work<ROWS>(a, load_request(a, r), plan).length;
        if (x < at + c) break;
        at += c;
      }
      s_walk[2 * w] = r;
      s_walk[2 * w + 1] = at;
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  // all columns are ours, so they start at 0
  if (tid == 0 && s_int[0] != 0) *abort = 1;

  // the pieces, for the roles that follow the loads
  uint32_t taken = 0;
  auto coming = [&](uint32_t i) {  // waits for piece i; false when there is none
    if (!__all_sync(0xffffffffu, bar_wait(b_piece + 8 * (i % AT_PIECES), (i / AT_PIECES) & 1, abort))) return false;
    return s_piece[i % AT_PIECES].valid != 0;
  };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) bar_arrive(b_taken + 8 * (taken % AT_PIECES));
    taken++;
  };

  // registers: 384 x 168 at launch = 128 x 104 + 256 x 200, where a softmax thread holds 128 scores
  if (warp < 4) {
    if (MODE == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0 || (warp == 3 && MODE != 2)) {
      // ---- loads, in the order of their use: K0 K1 V0 K2 V1 K3 ... with two tiles' scores, K0 V0 K1 V1 ... with one
      Walk<ROWS> walk;
      walk.plan = plan;
      walk.from = (blockIdx.x * WORKERS + ring) * plan.share;
      walk.to = min(total, walk.from + plan.share);
      walk.r = walk.from < total ? s_walk[2 * ring] : (int)a.R;
      walk.u = walk.from < total ? s_walk[2 * ring + 1] : total;
      walk.loaded = false;
      uint32_t at = 0, st = 0, ph = 0, filled = 0;  // pieces handed over; stage, its parity, stages filled (up to all)
      bool ok = true;
      auto hand = [&](const Piece& x) {
        ok = at < AT_PIECES || bar_wait(b_taken + 8 * (at % AT_PIECES), (at / AT_PIECES + 1) & 1, abort);
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (ok && lane == 0) {
          s_piece[at % AT_PIECES] = x;
          bar_arrive(b_piece + 8 * (at % AT_PIECES));
        }
        __syncwarp();
        at++;
      };
      // a box is 64 elements of a page's keys, at most 64 of them; a lane loads one box
      const int log2_box = min(a.log2_bs, 6), per_page = a.log2_bs - log2_box, ppt = KEYS >> log2_box;
      const int my_box = lane / HALVES, my_half = lane % HALVES;
      const uint32_t my_dst = s_ring + my_half * (KEYS * 128) + (my_box * 128 << log2_box);
      const uint32_t box_bytes = HALVES * 128u << log2_box;
      // block ids: a lane has box `window + lane`, and the one 32 further on
      struct Ids {
        int window, now, then;
      };
      int boxes = 0, h = 0;
      const int32_t* row = nullptr;
      auto id_of = [&](int b) { return b < boxes ? __ldg(row + (b >> per_page)) : 0; };
      auto load = [&](const CUtensorMap* map, Ids& ids, int tile) {
        const int box0 = tile * ppt;
        if (box0 >= ids.window + 32) {
          ids.window += 32;
          ids.now = ids.then;
          ids.then = id_of(ids.window + 32 + lane);
        }
        const int nb = max(0, min(ppt, boxes - box0));
        const int id = __shfl_sync(0xffffffffu, ids.now, (box0 + my_box) & 31);
        if (filled == NST) {
          ok = __all_sync(0xffffffffu, bar_wait(b_empty + 8 * st, ph ^ 1, abort)) != 0;
          if (!ok) return;
        } else {
          filled++;
        }
        if (elect_one()) bar_expect(b_full + 8 * st, nb * box_bytes);
        __syncwarp();
        if (my_box < nb)
          tma_load_4d(my_dst + st * L::STAGE, map, b_full + 8 * st, my_half * 64, per_page ? ((box0 + my_box) & 1) * 64 : 0, h, id);
        if (++st == NST) st = 0, ph ^= 1;
      };
      Piece nx;
      walk.next(a, nx);
      hand(nx);
      while (ok && nx.valid) {
        const int lo = nx.lo, hi = nx.hi;
        h = nx.h;
        boxes = (nx.keys + (1 << log2_box) - 1) >> log2_box;
        row = a.table + (int64_t)nx.r * a.table_stride;
        Ids k, v;
        k.window = (lo * ppt) & ~31;
        k.now = id_of(k.window + lane);
        k.then = id_of(k.window + 32 + lane);
        v = k;
        for (int t = lo; ok && t < min(hi, lo + BUFS); t++) load(&map_k, k, t);
        for (int t = lo; ok && t < hi; t++) {
          load(&map_v, v, t);
          // the next piece is known to the softmax, which asks for it in its last tile, before
          // more loads wait for it
          if (ok && t == lo) {
            walk.next(a, nx);
            hand(nx);
          }
          if (ok && t + BUFS < hi) load(&map_k, k, t + BUFS);
        }
      }
      // given up: the copies in flight land before the CTA ends
      if (*abort)
        for (uint32_t k = 0; k < filled; k++) {
          const uint32_t x = st + NST - filled + k;  // the stages filled last, oldest first
          for (uint32_t i = 0; i < 1u << 16 && !bar_try(b_full + 8 * (x % NST), x >= NST ? ph : ph ^ 1); i++) {}
        }
    } else if (warp == 1 || warp == 2) {
      // ---- products: the warp waits as one, one lane issues (with a branch of its own for
      // the lane every operand would be a divergent one: 120 cycles a product instead of 64)
      constexpr uint32_t KIND_S = mma_kind(BF, 128, KEYS, false), KIND_O = mma_kind(BF, 128, D, true);
      uint32_t st = 0, ph = 0, units = 0, nt = 0, turns = 0;  // stage, its parity; units, tiles, turns so far
      bool ok = true;
      const uint32_t q = mma_desc(s_q, 16);
      auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(bar, parity, abort)) != 0; };
      auto full = [&]() { return wait(b_full + 8 * st, ph); };
      auto advance = [&]() {
        if (++st == NST) st = 0, ph ^= 1;
      };
      auto scores = [&](uint32_t buf, uint32_t at) {  // S = Q K^T
        const uint32_t k = mma_desc(s_ring + at * L::STAGE, 16);
#pragma unroll
        for (int i = 0; i < D / 16; i++)
          mma_ss(stream * 256 + buf * KEYS, q + (((i >> 2) * (L::Q_ROWS * 128) + (i & 3) * 32) >> 4),
                 k + (((i >> 2) * (KEYS * 128) + (i & 3) * 32) >> 4), KIND_S, i > 0);
        mma_commit(b_s + 8 * buf);
        mma_commit(b_empty + 8 * at);
      };
      while (ok && coming(taken)) {
        const Piece& p = s_piece[taken % AT_PIECES];
        const int n = __shfl_sync(0xffffffffu, p.hi - p.lo, 0), rows = __shfl_sync(0xffffffffu, p.rows, 0);
        release();
        // Streams that share tiles take turns: products that come in together also end together, and
        // both streams then wait at once (2,048-token prompts: 211 us without, 200 with).
        const bool turn = MODE == 2 && rows > 128;
        if (MODE == 2 && stream * 128 >= rows) {  // no rows for this stream
          for (int i = 0; ok && i < 2 * n; i++, advance()) {
            ok = full();
            if (ok && lane == 0) bar_arrive(b_empty + 8 * st);
          }
          continue;
        }
        if (!(ok = wait(b_q, units & 1))) break;
        for (int t = 0; t < min(n, BUFS); t++, advance()) {
          if (!(ok = full())) break;
          tmem_fence_after();
          if (elect_one()) scores((nt + t) % BUFS, st);
          __syncwarp();
        }
        // the first output of a unit when the last one's has been read
        if (!ok || (units > 0 && !(ok = wait(b_free, (units + 1) & 1)))) break;
        for (int t = 0; t < n; t++, nt++) {
          // what is there early is waited for first: nothing but the weights is on the way from them to
          // the next scores
          const uint32_t sv = st, buf = nt % BUFS;
          if (!(ok = full())) break;
          advance();
          const uint32_t sk = st;
          const bool more = t + BUFS < n;
          if (more) {
            if (!(ok = full())) break;
            advance();
          }
          const uint32_t v = mma_desc(s_ring + sv * L::STAGE, KEYS * 128);
          if (!(ok = wait(b_p + 8 * buf, (nt / BUFS) & 1))) break;
          if (turn && (stream || turns > 0) && !(ok = wait(stream ? b_turn - 80 : b_turn + 80, (turns + 1 - stream) & 1))) break;
          turns += turn;
          tmem_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < KEYS / 16; i++)  // O += P V
              mma_ts(stream * 256 + 128, stream * 256 + buf * KEYS + i * 8, v + i * (2048 >> 4), KIND_O, t > 0 || i > 0);
            mma_commit(b_v);
            mma_commit(b_empty + 8 * sv);
            if (t == n - 1) mma_commit(b_o);
            if (more) scores(buf, sk);
            if (turn) bar_arrive(b_turn);
          }
          __syncwarp();
        }
        units++;
      }
      // given up: what was issued ends before tensor memory is freed
      if (*abort) {
        if (elect_one()) mma_commit(b_drain);
        __syncwarp();
        for (uint32_t i = 0; i < 1u << 16 && !bar_try(b_drain, 0); i++) {}
      }
    }
    __syncwarp();
  } else {
    if (MODE == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax
    const int wq = warp & 3, row = wq * 32 + lane;  // row = also its lane of tensor memory
    const uint32_t t_s = ((uint32_t)(wq * 32) << 16) + stream * 256, t_o = t_s + 128;
    const float c = a.scale_log2;
    const int me = blockIdx.x * 2 + stream;
    uint32_t nt = 0, units = 0, stages = 0;
    int joins = 0, join_first[2], join_pieces[2], join_rows[2], join_g[2], join_out[2];
    // A wait that gave up does not end the loops here (the next piece that does not come does):
    // what runs on is bounded, and its results are reported as an error.
    auto wait = [&](uint32_t bar, uint32_t parity) {
      bar_wait(bar, parity, abort);
      __syncwarp();
    };
    auto stream_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + stream) : "memory"); };
    constexpr int SKIP = MODE == 2 ? 128 : 0;  // rows of a unit before those of the second stream
    const int skip = stream * SKIP;
    // queries of the next piece, 16 bytes a copy, into 128-byte swizzled rows
    auto fetch = [&](uint32_t pc) {
      const Piece& x = s_piece[pc % AT_PIECES];
      const int row0 = x.row0 + skip, rows = min(128, x.rows - skip);
      const T* q = static_cast<const T*>(a.q) + x.t0 * a.q_stride + x.h * a.group * D;
#pragma unroll 4
      for (int i = row; i < rows * (D / 8); i += 128) {
        const int rr = i / (D / 8), ch = i % (D / 8), gr = row0 + rr, tok = gr / a.group;
        const T* src = q + tok * a.q_stride + (gr - tok * a.group) * D + ch * 8;
        const uint32_t dst = s_q + (ch >> 3) * (L::Q_ROWS * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
      }
    };
    auto fetched = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_async_smem();
      bar_arrive(b_q);
    };
    auto has_rows = [&](uint32_t pc) { return MODE != 2 || s_piece[pc % AT_PIECES].rows > skip; };
    bool more = coming(0);
    if (more && has_rows(0)) {
      fetch(0);
      fetched();
    }
    while (more) {
      const Piece& p = s_piece[taken % AT_PIECES];  // released at the unit's end: registers are short
      const int n = p.hi - p.lo, rows = min(128, p.rows - skip), open = p.open;
      const uint32_t ring0 = stages;  // its first stage
      stages += 2 * n;
      if (rows <= 0) {  // nothing for this stream
        if ((more = coming(taken + 1)) && has_rows(taken + 1)) {
          fetch(taken + 1);
          fetched();
        }
        release();
        continue;
      }
      const bool live = row < rows, active = wq * 32 < rows;  // the row's, the warp's
      const int gr = p.row0 + skip + row, tok = live ? gr / a.group : 0;
      Seen seen;
      seen.tree = a.mask != nullptr;
      seen.ctx = p.ctx;
      seen.last = p.valid == 2 ? p.ctx + tok : -1;
      seen.mask = 0;
      if (seen.tree && live && p.valid == 2) {
        seen.mask = (uint64_t)a.mask[p.t0 + tok];
        if (p.n < 64) seen.mask &= (1ull << p.n) - 1;
      }
      float m = -INFINITY, mc = 0.f, l = 0.f, l_full = 0.f;  // mc = m c - UP, or 0 while the row has seen nothing
      const int lo = p.lo;
      const uint64_t c2 = pair64(c, c);

      // One tile.  Nearly all are seen by every row; where the softmax is the bound (MODE 2) those have a
      // body of their own.
      auto tile = [&](int t, auto some_hidden) {
        const int k0 = (lo + t) * KEYS;
        const bool hidden = decltype(some_hidden)::value && (MODE == 2 || k0 + KEYS > open);
        if (hidden) {
          // Values of keys past the request's end become 0; so do infinities and NaN of
          // keys that only some rows see: 0 * inf in a product would reach the others.
          // (Rows that do see them get them back below.)  Streams that share a tile leave it to the first.
          if (MODE != 2 || stream == 0) {
            const uint32_t at = ring0 + (BUFS == 1 ? 2 * t + 1 : n == 1 ? 1 : t == n - 1 ? 2 * n - 1 : 2 * t + 2);
            wait(b_full + 8 * (at % NST), (at / NST) & 1);
            constexpr int PARTS = 128 / KEYS;  // threads of a row
            const int kr = row % KEYS, part = row / KEYS, key = k0 + kr;
            if (key >= open) {
              uint8_t* v = smem + (s_ring - base) + (at % NST) * L::STAGE + kr * 128;
              bool bad = false;
#pragma unroll 4
              for (int i = part * (D / 8 / PARTS); i < (part + 1) * (D / 8 / PARTS); i++) {
                uint4* x = reinterpret_cast<uint4*>(v + (i >> 3) * (KEYS * 128) + (((i & 7) ^ (kr & 7)) << 4));
                if (key >= p.len) {
                  *x = make_uint4(0, 0, 0, 0);
                } else {
                  uint4 y = *x;
                  uint32_t* z = reinterpret_cast<uint32_t*>(&y);
                  if (nonfinite2<T>(z[0]) | nonfinite2<T>(z[1]) | nonfinite2<T>(z[2]) | nonfinite2<T>(z[3])) {
                    bad = true;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                      const uint32_t b = nonfinite2<T>(z[e]);
                      if (b & 0x8000u) z[e] &= 0xffff0000u;
                      if (b & 0x80000000u) z[e] &= 0x0000ffffu;
                    }
                    *x = y;
                  }
                }
              }
              if (bad) s_bad[taken & 7] = 1;
            }
            fence_async_smem();
          }
          if (MODE == 2 && p.rows > 128) asm volatile("bar.sync 3, 256;" ::: "memory");
        }
        const uint32_t buf = nt % BUFS;
        wait(b_s + 8 * buf, (nt / BUFS) & 1);
        tmem_fence_after();
        uint32_t s[KEYS];
        if (active) {
#pragma unroll
          for (int i = 0; i < KEYS; i += 32) tmem_ld32(s + i, t_s + buf * KEYS + i);
          tmem_wait_ld();
          if (hidden) {
#pragma unroll
            for (int i = 0; i < KEYS / 32; i++) {
              const uint32_t w = seen.bits(k0 + 32 * i);
#pragma unroll
              for (int e = 0; e < 32; e++)
                if (!((w >> e) & 1)) s[32 * i + e] = 0xff800000u;
            }
          }
          float top[4];
#pragma unroll
          for (int i = 0; i < 4; i++) top[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
          for (int i = 8; i < KEYS; i += 2)
            top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]);
          const bool grow = t == 0 || (live && mx > m && !((mx - m) * c <= 8.f));
          if (__any_sync(0xffffffffu, grow)) {
            if (t > 0) {
              // the products of the tile before may still run
              wait(b_v, (nt + 1) & 1);
              tmem_fence_after();
              const float f = grow ? exp2_fast((m - mx) * c) : 1.f;
#pragma unroll 1
              for (int i = 0; i < D / 32; i++) {
                uint32_t o[32];
                tmem_ld32(o, t_o + 32 * i);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(t_o + 32 * i, o);
              }
              l *= f;
              l_full *= f;
            }
            if (grow) {
              m = mx;
              mc = m == -INFINITY ? 0.f : fmaf(m, c, -UP);
            }
          }
          const uint64_t mc2 = pair64(-mc, -mc);
          float sum[4] = {0.f, 0.f, 0.f, 0.f};  // of the rounded weights, which the product has
          uint64_t full[2] = {0, 0};            // of the weights
#pragma unroll
          for (int i = 0; i < KEYS / 64; i++) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; e++) {
              const float2 x = unpair64(fma2(pair64(s[64 * i + 2 * e], s[64 * i + 2 * e + 1]), c2, mc2));
              const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y);
              if (LSE) full[e & 1] = add2(full[e & 1], pair64(p0, p1));
              w[e] = pack2<T>(p0, p1);
              add_halves(sum[2 * (e & 1)], sum[2 * (e & 1) + 1], w[e], BF);
            }
            tmem_st32(t_s + buf * KEYS + 32 * i, w);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          if (LSE) {
            const float2 l2 = unpair64(add2(full[0], full[1]));
            l_full += l2.x + l2.y;
          }
          tmem_wait_st();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(b_p + 8 * buf);
        nt++;
      };
      int clear = 0;
      if constexpr (MODE == 2) {
        clear = max(0, min(n, open / KEYS - lo));
#pragma unroll 1
        for (int t = 0; t < clear; t++) tile(t, std::false_type());
      }
#pragma unroll 1
      for (int t = clear; t < n; t++) tile(t, std::true_type());
      // the queries have been read for the last time: the next ones come in under the last products
      more = coming(taken + 1);
      if (more && has_rows(taken + 1)) {
        fetch(taken + 1);
        fetched();
      }
      wait(b_o, units & 1);
      tmem_fence_after();

      const bool whole = p.pieces == 1;
      const bool bad = s_bad[taken & 7] != 0;
      float* part = part_at<D>(a.part, me, p.lo == 0);
      const int64_t o_at = (int64_t)(p.t0 + tok) * a.hq + p.h * a.group + (gr - tok * a.group);
      if (active) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t x[32];
          tmem_ld32(x, t_o + d);
          tmem_wait_ld();
          if (live) {
            float o[32];
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = l == 0.f ? 0.f : __uint_as_float(x[e]) * inv;
            if (whole) {
              T* dst = static_cast<T*>(a.out) + o_at * D + d;
#pragma unroll
              for (int e = 0; e < 4; e++)
                *reinterpret_cast<uint4*>(dst + 8 * e) =
                    make_uint4(pack2<T>(o[8 * e], o[8 * e + 1]), pack2<T>(o[8 * e + 2], o[8 * e + 3]),
                               pack2<T>(o[8 * e + 4], o[8 * e + 5]), pack2<T>(o[8 * e + 6], o[8 * e + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(part) + (d / 4) * 128 + row;
#pragma unroll
              for (int e = 0; e < 8; e++) __stcg(dst + e * 128, make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
            }
          }
          __syncwarp();
        }
        if (live) {
          if (!whole) {
            __stcg(part + 128 * D + row, l == 0.f ? -INFINITY : mc + log2f(l));
            if (LSE) __stcg(part + 128 * D + 128 + row, l == 0.f ? 1.f : l_full / l);
          } else if (LSE && a.lse) {
            a.lse[o_at] = l == 0.f ? -INFINITY : (mc + log2f(l_full)) * 0.69314718055994531f;
          }
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(b_free);
      // two pieces ahead; streams that share it are at most AT_PIECES apart
      if (row == 0 && (MODE != 2 || stream == 0)) s_bad[(taken + 2) & 7] = 0;
      if (bad && live) {
        // the values taken out above, for the rows that see them: any weight makes them infinite or NaN
        const int to = min(p.len, p.hi * KEYS);
        for (int j = max(open, p.lo * KEYS); j < to; j++) {
          const int64_t id = a.table[(int64_t)p.r * a.table_stride + (j >> a.log2_bs)];
          if (!seen.has(j) || id < 0 || id >= a.n_blocks) continue;
          const T* v = static_cast<const T*>(a.v) + id * a.s_block + p.h * a.s_head + (j & ((1 << a.log2_bs) - 1)) * a.s_token;
          for (int d = 0; d < D; d++) {
            const float y = (float)v[d];
            if (fabsf(y) < INFINITY) continue;
            if (whole) {
              T* dst = static_cast<T*>(a.out) + o_at * D + d;
              *dst = (T)((float)*dst + y);
            } else {
              float* dst = part + (d / 4) * 512 + row * 4 + (d & 3);
              __stcg(dst, __ldcg(dst) + y);
            }
          }
        }
      }
      if (!whole) {
        __threadfence();
        stream_sync();
        const int key = MODE == 2 ? p.first * 2 + stream : p.first;
        if (row == 0) atomicAdd(a.counters + 2 * key, 1u);
        if (joins < 2) {
          join_first[joins] = key;
          join_pieces[joins] = p.pieces;
          join_rows[joins] = rows;
          join_g[joins] = p.row0 + skip;
          join_out[joins] = p.t0 * a.hq + p.h * a.group;
          joins++;
        }
      }
      release();
      units++;
    }
    // The streams that a unit is divided over join it together, each some of its
    // outputs, the pieces always in the same order.  They wait for one another:
    // the launch is cooperative, so all are resident, and each ends its pieces first.
    for (int k = 0; k < joins && !*abort; k++) {
      constexpr int STEP = MODE == 2 ? 2 : 1;  // from one piece's stream to the next one's
      const int key = join_first[k], np = join_pieces[k], mine = (me - key) / STEP, rows = join_rows[k];
      if (row == 0) {
        const volatile unsigned* done = a.counters + 2 * key;
        for (uint32_t i = 0; *done < (unsigned)np && !*abort; i++) {
          if (i > 1u << 24) *abort = 1;
          __nanosleep(20);
        }
        __threadfence();
      }
      stream_sync();
      if (*abort) break;
      // an item is four columns of a row; G lanes share its pieces, at most 8 at a time each
      int G = 1;
      while (G < 32 && G * 8 < np) G *= 2;
      const int items = rows * (D / 4), each = (items + np - 1) / np, to = min(items, (mine + 1) * each), g = lane & (G - 1);
      for (int i = mine * each + row / G; i - row / G < to; i += 128 / G) {
        const bool in = i < to;
        const int rr = in ? i % rows : 0, ch = in ? i / rows : 0;
        float top = -INFINITY, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = g; j0 < np; j0 += 8 * G) {
          float e[8];
          float4 x[8];
#pragma unroll
          for (int j = 0; j < 8; j++) {
            const int pc = j0 + j * G;
            const float* src = part_at<D>(a.part, key + pc * STEP, pc == 0);
            e[j] = pc < np ? __ldcg(src + 128 * D + rr) : -INFINITY;
            x[j] = pc < np ? __ldcg(reinterpret_cast<const float4*>(src) + ch * 128 + rr) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          float up = top;
#pragma unroll
          for (int j = 0; j < 8; j++) up = fmaxf(up, e[j]);
          const float f = top == -INFINITY ? 0.f : exp2_fast(top - up);
          sum *= f;
          o.x *= f; o.y *= f; o.z *= f; o.w *= f;
          top = up;
#pragma unroll
          for (int j = 0; j < 8; j++) {
            if (e[j] == -INFINITY) continue;  // a piece without weight
            const float w = exp2_fast(e[j] - top);
            sum += w;
            o.x = fmaf(w, x[j].x, o.x);
            o.y = fmaf(w, x[j].y, o.y);
            o.z = fmaf(w, x[j].z, o.z);
            o.w = fmaf(w, x[j].w, o.w);
          }
        }
        for (int d = 1; d < G; d *= 2) {
          const float t2 = __shfl_xor_sync(0xffffffffu, top, d), up = fmaxf(top, t2);
          const float f = top == -INFINITY && sum == 0.f ? 0.f : top == up ? 1.f : exp2_fast(top - up);
          sum *= f;
          o.x *= f; o.y *= f; o.z *= f; o.w *= f;
          top = up;
          sum += __shfl_xor_sync(0xffffffffu, sum, d);
          o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
          o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
          o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
          o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
        }
        if (in && g == 0) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const int gr = join_g[k] + rr, tk = gr / a.group;
          const int64_t at = (int64_t)join_out[k] + (int64_t)tk * a.hq + (gr - tk * a.group);
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + ch * 4) =
              make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
          if (LSE && a.lse && ch == 0) {
            float full = 0.f;
#pragma unroll 1
            for (int pc = 0; pc < np; pc++) {
              const float* src = part_at<D>(a.part, key + pc * STEP, pc == 0) + 128 * D + rr;
              const float e = __ldcg(src);
              if (e != -INFINITY) full = fmaf(exp2_fast(e - top), __ldcg(src + 128), full);
            }
            a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(full)) * 0.69314718055994531f;
          }
        }
      }
      stream_sync();
      if (row == 0 && atomicAdd(a.counters + 2 * key + 1, 1u) == (unsigned)np - 1) {
        a.counters[2 * key] = 0;  // all have seen it
        a.counters[2 * key + 1] = 0;
      }
    }
  }
  // over whatever was met before: tk_kv_status clears the counters for this one only
  if (*abort && lane == 0) {
    atomicExch(&a.status->code, TK_E_TIMEOUT);
    a.status->request = -1;
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    tmem_free(0);
  }
}

template <class T, int D, int MODE, bool LSE>
static cudaError_t attend_launch(const AttendArgs& a, const tk_kv_cache* cache, int grid, cudaStream_t st) {
  constexpr int bytes = AttendShape<D, MODE>::TOTAL;
  static bool set[64];  // by device
  if (cache->device >= 64 || !set[cache->device]) {
    const cudaError_t e = cudaFuncSetAttribute(k_kv_attend<T, D, MODE, LSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (cache->device < 64) set[cache->device] = true;
  }
  cudaLaunchAttribute coop;
  coop.id = cudaLaunchAttributeCooperative;
  coop.val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(AT_THREADS);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cfg.attrs = &coop;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv_attend<T, D, MODE, LSE>, a, cache->map_k, cache->map_v);
}

template <class T, int D>
static cudaError_t attend_pick(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  if (rows <= 32) return attend_launch<T, D, 0, true>(a, cache, grid, st);
  if (rows <= 128) return attend_launch<T, D, 1, true>(a, cache, grid, st);
  return a.lse ? attend_launch<T, D, 2, true>(a, cache, grid, st) : attend_launch<T, D, 2, false>(a, cache, grid, st);
}

}  // namespace tk

static int attend_arg(const char* where, const char* what) {
  tk_set_error("%s: %s", where, what);
  return TK_E_ARG;
}

extern "C" int tk_kv_workspace_create(tk_kv_workspace** out) {
  using namespace tk;
  const char* where = "tk_kv_workspace_create";
  if (!out) return attend_arg(where, "null pointer");
  *out = nullptr;
  tk_kv_workspace* ws = new (std::nothrow) tk_kv_workspace();
  if (!ws) {
    tk_set_error("%s: out of memory", where);
    return TK_E_NOMEM;
  }
  cudaError_t e = cudaGetDevice(&ws->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&ws->sms, cudaDevAttrMultiProcessorCount, ws->device);
  // one allocation: the partial outputs of two pieces of every stream, its counters, the status
  const size_t part = sizeof(float) * 2 * 2 * 128 * (128 + 2) * (size_t)ws->sms,
               counters = sizeof(unsigned) * 2 * 2 * (size_t)ws->sms;
  uint8_t* mem = nullptr;
  if (e == cudaSuccess) e = cudaMalloc(&mem, part + counters + 64 + sizeof(KvStatus));
  if (e == cudaSuccess) {
    ws->part = reinterpret_cast<float*>(mem);
    ws->counters = reinterpret_cast<unsigned*>(mem + part);
    ws->status = reinterpret_cast<KvStatus*>(mem + (part + counters + 63) / 64 * 64);
    e = cudaMemset(ws->counters, 0, counters + 64 + sizeof(KvStatus));
    // a first call on a stream that does not wait for the legacy one would find them as they were
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) {
    tk_set_error("%s: %s", where, cudaGetErrorString(e));
    tk_kv_workspace_free(ws);
    return e == cudaErrorMemoryAllocation ? TK_E_NOMEM : TK_E_CUDA;
  }
  *out = ws;
  return TK_OK;
}

extern "C" void tk_kv_workspace_free(tk_kv_workspace* ws) {
  if (!ws) return;
  cudaFree(ws->part);
  delete ws;
}

extern "C" int tk_kv_status(tk_kv_workspace* ws, int64_t* h_request, void* cuda_stream) {
  using namespace tk;
  if (h_request) *h_request = -1;
  if (!ws) return attend_arg("tk_kv_status", "null workspace");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != ws->device)
    return attend_arg("tk_kv_status", "the current device is not the workspace's");
  KvStatus s = {};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  cudaError_t e = cudaMemcpyAsync(&s, ws->status, sizeof(s), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && s.code) e = cudaMemsetAsync(ws->status, 0, sizeof(s), st);
  // a call that gave up may have left counts behind
  if (e == cudaSuccess && s.code == TK_E_TIMEOUT) e = cudaMemsetAsync(ws->counters, 0, sizeof(unsigned) * 4 * ws->sms, st);
  if (e != cudaSuccess) {
    tk_set_error("tk_kv_status: %s", cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  if (s.code) {
    if (h_request) *h_request = s.request;
    if (s.code == TK_E_TIMEOUT) tk_set_error("tk_kv_attend: a wait on the device gave up");
    else if (s.request < 0) tk_set_error("tk_kv_attend: more work than one call takes, or offsets that contradict each other");
    else tk_set_error("tk_kv_attend: request %lld: lengths outside the call's limits", (long long)s.request);
  }
  return s.code;
}

extern "C" int tk_kv_attend(const tk_kv_cache* cache, tk_kv_workspace* ws, const void* d_q, int64_t q_stride,
                            int n_q_heads, const int64_t* d_off, int64_t R, int64_t T, int64_t max_new,
                            const int32_t* d_len, const int32_t* d_table, int64_t table_stride, int64_t table_width,
                            const int64_t* d_mask, float scale, void* d_out, float* d_lse, void* cuda_stream) {
  using namespace tk;
  const char* where = "tk_kv_attend";
  if (!cache || !ws) return attend_arg(where, "null cache or workspace");
  if (ws->device != cache->device) return attend_arg(where, "cache and workspace are on different devices");
  if (cache->head_dim != 64 && cache->head_dim != 128) return attend_arg(where, "head_dim is neither 64 nor 128");
  if (n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % cache->n_heads)
    return attend_arg(where, "n_q_heads is no multiple of the cache's heads up to 1,024");
  if (R < 0 || T < 0 || R > 1 << 20 || T > 1 << 26 || max_new < 0 || table_width < 0 || table_stride < table_width)
    return attend_arg(where, "bad size");
  if (q_stride < (int64_t)n_q_heads * cache->head_dim || q_stride % 8)
    return attend_arg(where, "q_stride is below a token's elements or no multiple of 8");
  if (!(scale > 0.f && scale < 1e38f)) return attend_arg(where, "scale is not a positive number below 1e38");
  if (T * n_q_heads > INT32_MAX) return attend_arg(where, "T times n_q_heads is above 2^31");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != cache->device) return attend_arg(where, "the current device is not the cache's");
  if (T == 0) return TK_OK;
  if (!d_q || !d_out || (R > 0 && (!d_off || !d_len || (table_width > 0 && !d_table)))) return attend_arg(where, "null pointer");
  if ((((uintptr_t)d_q | (uintptr_t)d_out) & 15) != 0) return attend_arg(where, "a buffer is not 16-byte aligned");
  const int group = n_q_heads / cache->n_heads;
  AttendArgs a = {d_q, q_stride, n_q_heads, cache->n_heads, group, d_off, R, T, max_new, d_len, d_table, table_stride,
                  table_width, d_mask, scale * 1.4426950408889634f, d_out, d_lse, ws->status,
                  cache->v, cache->n_blocks, cache->stride[0], cache->stride[1],
                  cache->stride[2], cache->log2_block, ws->part, ws->counters};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const int64_t rows = std::min(max_new, T) * group;  // of a request and key head
  cudaError_t e;
  if (cache->type == TK_BF16)
    e = cache->head_dim == 64 ? attend_pick<__nv_bfloat16, 64>(a, cache, rows, ws->sms, st)
                              : attend_pick<__nv_bfloat16, 128>(a, cache, rows, ws->sms, st);
  else
    e = cache->head_dim == 64 ? attend_pick<__half, 64>(a, cache, rows, ws->sms, st)
                              : attend_pick<__half, 128>(a, cache, rows, ws->sms, st);
  if (e != cudaSuccess) {
    tk_set_error("%s: %s", where, cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  return TK_OK;
}
