// tk_attend.cu -- attention of new and drafted tokens over the paged cache
// (tk_kv_attend): o = sum_j softmax_j(scale q.k_j) v_j over the keys j that a
// token sees.
//
// The query rows of one request and key head (tokens x query heads of that key
// head) are the rows of the products S = Q K^T and O = P V on the 5th-generation
// tensor cores; 128 rows are one tile whether they are all in use or not: a
// tile's two products take about 1,000 cycles against the 2,850 that its
// 64 KB of keys and values take from HBM (head_dim 128), so padding costs nothing while
// memory is the bound.  Keys come in tiles of 128.  With a running maximum m and sum l,
//   p_j = 2^(c (s_j - m)), c = scale log2(e),  l += sum p_j,  O += P V,
// and O is rescaled in tensor memory only when m grows by more than 2^8 in p
// (p and l are relative to the same m, so the quotient is exact either way).
// S, m, l and O are fp32; P is rounded to the cache's type, which the tensor
// cores ask for: an error of half an ulp in each weight.
#include <algorithm>
#include <new>

#include "tk_blackwell.cuh"
#include "tk_kv.cuh"

namespace tk {

constexpr int AT_KEYS = 128;      // keys of a tile
constexpr int AT_THREADS = 384;   // 4 warps of producer, products and none; 2 x 4 softmax warps
constexpr int AT_UNIT_COST = 1;   // what starting a unit costs, in tiles
constexpr int AT_MIN_SHARE = 4;   // least share of a CTA, in tiles

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
  const uint8_t* v;
  int64_t n_blocks, s_block, s_head, s_token;
  int log2_bs;
  float* part;         // partial outputs, see part_at
  unsigned* counters;  // [gridDim.x] pieces of a divided unit that are done, by its first CTA
};

// A request as the schedule sees it.
struct Request {
  int64_t t0;   // its first row of q
  int32_t n, ctx, len;
  int tiles_m;  // row tiles
  bool good;
};

template <int ROWS>
__device__ __forceinline__ Request load_request(const AttendArgs& a, int64_t r) {
  Request q;
  q.t0 = a.off[r];
  const int64_t n = a.off[r + 1] - q.t0, len = a.len[r];
  q.good = n >= 0 && n <= a.max_new && (!a.mask || n <= KV_TREE_MAX) && len >= n && len <= a.table_width << a.log2_bs &&
           q.t0 >= 0 && q.t0 + n <= a.T;
  // rows that cannot be taken are written as zeros, inside the output whatever the offsets say
  if (q.t0 < 0) q.t0 = 0;
  q.n = (int32_t)max((int64_t)0, min(n, a.T - q.t0));
  q.len = q.good ? (int32_t)len : 0;
  q.ctx = q.good ? (int32_t)(len - n) : 0;
  q.tiles_m = (int)(((int64_t)q.n * a.group + ROWS - 1) / ROWS);
  return q;
}

// Keys that row tile m reads, and their tiles (at least one: it writes the rows).
template <int ROWS>
__device__ __forceinline__ int unit_keys(const AttendArgs& a, const Request& q, int m) {
  if (a.mask || !q.good) return q.len;
  const int64_t last = min((int64_t)q.n * a.group, (int64_t)(m + 1) * ROWS) - 1;
  return q.ctx + (int)(last / a.group) + 1;
}
__device__ __forceinline__ int key_tiles(int keys) { return max(1, (keys + AT_KEYS - 1) / AT_KEYS); }

template <int ROWS>
__device__ __forceinline__ int64_t request_cost(const AttendArgs& a, const Request& q) {
  int64_t c = 0;
  if (a.mask || !q.good) c = (int64_t)q.tiles_m * (key_tiles(q.len) + AT_UNIT_COST);
  else
    for (int m = 0; m < q.tiles_m; m++) c += key_tiles(unit_keys<ROWS>(a, q, m)) + AT_UNIT_COST;
  return c * a.hk;
}

// The work is one line of units (request, row tile, key head), each AT_UNIT_COST
// + its key tiles long; CTA c takes [c * share, (c + 1) * share) of it, so that
// a long cache is divided over CTAs and short ones are gathered in one.  A warp
// walks the CTA's part of the line and hands the pieces to the other roles.
struct Piece {
  int t0, r, h;        // first row of q, request, key head
  int row0, rows;      // rows of the unit among the request's tokens x group
  int n, ctx, len;     // of the request; ctx = len = 0 if it cannot be taken
  int open;            // keys that every row of the unit sees
  int keys, lo, hi;    // keys of the unit; tiles of this piece
  int first, pieces;   // the CTA with the unit's tile 0; CTAs it is divided over
  int valid;           // 0 = no more
};
constexpr int AT_PIECES = 4;  // handed over ahead

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

template <int D, int TILES>
struct AttendSmem {
  static constexpr int STAGE = AT_KEYS * D * 2;
  static constexpr int Q = TILES * 128 * D * 2;
  static constexpr int STAGES = D == 64 ? 12 : (TILES == 1 ? 6 : 5);
  static constexpr int BARS = Q + STAGES * STAGE;
  static constexpr int SMALL = BARS + 8 * (2 * STAGES + 8 + 2 * AT_PIECES);
  // tmem, abort, non-finite values (2), last piece, start of the walk (2 x 8); sums of the warps; pieces; then m and l
  // of both streams
  static constexpr int PIECES = SMALL + 48 + 8 * (AT_THREADS / 32);
  static constexpr int ML = PIECES + AT_PIECES * (int)sizeof(Piece);
  static constexpr int TOTAL = ML + 2 * 128 * 8;
  static_assert(TOTAL <= 227 * 1024, "shared memory of one CTA");
};

// Partial output of a piece: [row][D] normalised, then [row] log2 of the sum.
// A CTA has at most two: slot 1 = it holds the unit's first tile.
template <int D, int ROWS>
__device__ __forceinline__ float* part_at(const AttendArgs& a, int64_t cta, int slot) {
  return a.part + (cta * 2 + slot) * (ROWS * (D + 1));
}

// Warp 0 loads, warp 1 issues the products, warps 4-7 and 8-11 are two softmax
// streams with scores and outputs of their own in tensor memory (S 0-127 and
// 128-255, O from 256 and 384; P over the first half of S).  TILES = 1: both
// work on the same 128 rows, one on the even and one on the odd key tiles, and are
// joined at the end.  TILES = 2: each has 128 rows, both read every tile.  While
// one stream is in its softmax the other's products run.
template <class T, int D, int TILES>
__global__ void __launch_bounds__(AT_THREADS, 1)
k_kv_attend(const AttendArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using L = AttendSmem<D, TILES>;
  constexpr int ROWS = TILES * 128, HALVES = D / 64, NST = L::STAGES;
  constexpr bool BF = Pair<T>::BF;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle goes by address bits
  const uint32_t base = smem_addr(smem), s_q = base, s_ring = base + L::Q;
  const uint32_t b_full = base + L::BARS, b_empty = b_full + 8 * NST, b_q = b_empty + 8 * NST, b_s = b_q + 8, b_p = b_s + 16,
                 b_o = b_p + 16, b_drain = b_o + 8, b_piece = b_drain + 8, b_taken = b_piece + 8 * AT_PIECES;
  int* small = reinterpret_cast<int*>(smem + L::SMALL);
  volatile int* abort = small + 1;
  volatile int* s_bad = small + 2;    // [2] non-finite values among the drafted tokens, by parity of the unit
  volatile int* s_last = small + 4;
  int64_t* s_walk = reinterpret_cast<int64_t*>(small + 8);  // first request, where it starts
  int64_t* s_sum = reinterpret_cast<int64_t*>(small + 12);
  Piece* s_piece = reinterpret_cast<Piece*>(smem + L::PIECES);
  float2* s_ml = reinterpret_cast<float2*>(smem + L::ML);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (base & 1023) {  // never: the swizzle would not hold
    if (tid == 0) a.status->code = TK_E_CUDA;
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NST; i++) {
      bar_init(b_full + 8 * i, 1);
      bar_init(b_empty + 8 * i, 1);
    }
    bar_init(b_q, 256);
    bar_init(b_s, 1);
    bar_init(b_s + 8, 1);
    bar_init(b_p, 4);
    bar_init(b_p + 8, 4);
    bar_init(b_o, 1);
    bar_init(b_drain, 1);
    for (int i = 0; i < AT_PIECES; i++) {
      bar_init(b_piece + 8 * i, 1);
      bar_init(b_taken + 8 * i, 10);  // loads, products, 8 softmax warps
    }
    fence_bar_init();
    small[1] = small[2] = small[3] = 0;
  }
  if (warp == 1) tmem_alloc(smem_addr(small));

  // where this CTA starts: the requests' costs added up, each thread a run of them
  int64_t share, x0, total;
  {
    const int64_t per = (a.R + AT_THREADS - 1) / AT_THREADS;
    const int64_t r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
    int64_t sum = 0;
    for (int64_t r = r0; r < r1; r++) {
      const Request q = load_request<ROWS>(a, r);
      if (!q.good && blockIdx.x == 0 && atomicCAS(&a.status->code, 0, TK_E_LIMIT) == 0) a.status->request = r;
      sum += request_cost<ROWS>(a, q);
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t before = incl - sum;
    total = 0;
    for (int w = 0; w < AT_THREADS / 32; w++) {
      const int64_t y = s_sum[w];
      if (w < warp) before += y;
      total += y;
    }
    share = max((int64_t)AT_MIN_SHARE, (total + gridDim.x - 1) / gridDim.x);
    x0 = blockIdx.x * share;
    if (x0 >= before && x0 < before + sum) {
      int64_t r = r0, at = before;
      for (; r < r1 - 1; r++) {
        const int64_t c = request_cost<ROWS>(a, load_request<ROWS>(a, r));
        if (x0 < at + c) break;
        at += c;
      }
      s_walk[0] = r;
      s_walk[1] = at;
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(small);
  // the next piece, for a whole role; false at the end
  uint32_t taken = 0;
  Piece p;
  auto next = [&]() {
    if (!bar_wait(b_piece + 8 * (taken % AT_PIECES), (taken / AT_PIECES) & 1, abort)) return false;
    p = s_piece[taken % AT_PIECES];
    return p.valid != 0;
  };
  auto release = [&]() { bar_arrive(b_taken + 8 * (taken++ % AT_PIECES)); };

  // registers: 384 x 168 at launch = 128 x 56 + 256 x 224
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 0) {
    // ---- loads: one box per page and 64 elements; lanes hold the ids of 32 pages, and of the next 32
    uint32_t pos = 0;
    const int ppt = AT_KEYS >> a.log2_bs;  // pages of a tile
    bool ok = true;
    while (ok && __all_sync(0xffffffffu, next())) {
      __syncwarp();
      if (lane == 0) release();
      else taken++;
      const int n = p.hi - p.lo, pages = (p.keys + (1 << a.log2_bs) - 1) >> a.log2_bs;
      const int32_t* row = a.table + (int64_t)p.r * a.table_stride;
      int window = (p.lo * ppt) & ~31;
      // keys run ahead of values: two id windows each
      int ids_k = window + lane < pages ? row[window + lane] : 0, win_k = window;
      int nxt_k = window + 32 + lane < pages ? row[window + 32 + lane] : 0;
      int ids_v = ids_k, nxt_v = nxt_k, win_v = window;
      const int loads = 2 * n;
      for (int i = 0; i < loads; i++, pos++) {
        // order of use: TILES 1: K0 K1 V0 K2 V1 K3 ...; TILES 2: K0 V0 K1 V1 ...
        bool value;
        int t;
        if (TILES == 2) {
          value = i & 1;
          t = i >> 1;
        } else {
          const int lead = min(n, 2);
          if (i < lead) value = false, t = i;
          else if (i == loads - 1) value = true, t = n - 1;
          else value = ((i - lead) & 1) == 0, t = value ? (i - lead) >> 1 : ((i - lead) >> 1) + 2;
        }
        const int page0 = (p.lo + t) * ppt;
        if (value) {
          if (page0 >= win_v + 32) {
            win_v += 32;
            ids_v = nxt_v;
            nxt_v = win_v + 32 + lane < pages ? row[win_v + 32 + lane] : 0;
          }
        } else if (page0 >= win_k + 32) {
          win_k += 32;
          ids_k = nxt_k;
          nxt_k = win_k + 32 + lane < pages ? row[win_k + 32 + lane] : 0;
        }
        const int np = max(0, min(ppt, pages - page0));
        const uint32_t st = pos % NST, dst = s_ring + st * L::STAGE;
        ok = pos < NST || bar_wait(b_empty + 8 * st, (pos / NST + 1) & 1, abort);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (lane == 0) bar_expect(b_full + 8 * st, (uint32_t)np * (HALVES * 128u << a.log2_bs));
        const int src = (page0 + lane) & 31;
        const int id = __shfl_sync(0xffffffffu, value ? ids_v : ids_k, src);
        __syncwarp();
        if (lane < np) {
#pragma unroll
          for (int s = 0; s < HALVES; s++)
            tma_load_4d(dst + s * (AT_KEYS * 128) + (lane * 128 << a.log2_bs), value ? &map_v : &map_k, b_full + 8 * st, s * 64,
                        0, p.h, id);
        }
      }
    }
    // given up: the copies in flight land before the CTA ends
    if (*abort)
      for (uint32_t k = pos > NST ? pos - NST : 0; k < pos; k++)
        for (uint32_t i = 0; i < 1u << 16 && !bar_try(b_full + 8 * (k % NST), (k / NST) & 1); i++) {}
  } else if (warp == 1) {
    // ---- products, issued by one lane
    if (lane == 0) {
      constexpr uint32_t KIND_S = mma_kind(BF, 128, AT_KEYS, false), KIND_O = mma_kind(BF, 128, D, true);
      uint32_t pos = 0, units = 0, np[2] = {0, 0};
      bool ok = true;
      auto scores = [&](int stream, uint32_t at, int tile) {  // S = Q K^T
        const uint32_t k = mma_desc(s_ring + (at % NST) * L::STAGE, 16), q = mma_desc(s_q + tile * (128 * D * 2), 16);
#pragma unroll
        for (int i = 0; i < D / 16; i++) {
          const uint32_t o = (i >> 2) * (128 * 128) + (i & 3) * 32;
          mma_ss(tmem + stream * 128, q + (o >> 4), k + (o >> 4), KIND_S, i > 0);
        }
      };
      auto outputs = [&](int stream, uint32_t at, bool add) {  // O += P V
        const uint32_t v = mma_desc(s_ring + (at % NST) * L::STAGE, AT_KEYS * 128);
#pragma unroll
        for (int i = 0; i < AT_KEYS / 16; i++)
          mma_ts(tmem + 256 + stream * 128, tmem + stream * 128 + i * 8, v + i * (2048 >> 4), KIND_O,
                 add || i > 0);
      };
      auto full = [&](uint32_t at) { return bar_wait(b_full + 8 * (at % NST), (at / NST) & 1, abort); };
      auto weights = [&](int stream) { return bar_wait(b_p + 8 * stream, np[stream]++ & 1, abort); };
      while (ok && next()) {
        release();
        const int n = p.hi - p.lo;
        ok = bar_wait(b_q, units & 1, abort);
        units++;
        if (!ok) break;
        tmem_fence_after();
        if (TILES == 1) {
          for (int t = 0; ok && t < min(n, 2); t++) {
            if (!(ok = full(pos))) break;
            tmem_fence_after();
            scores(t, pos, 0);
            mma_commit(b_empty + 8 * (pos % NST));
            mma_commit(b_s + 8 * t);
            pos++;
          }
          for (int t = 0; ok && t < n; t++) {
            const int s = t & 1;
            if (!(ok = full(pos) && weights(s))) break;
            tmem_fence_after();
            outputs(s, pos, t >= 2);
            mma_commit(b_empty + 8 * (pos % NST));
            pos++;
            if (t + 2 < n) {
              if (!(ok = full(pos))) break;
              tmem_fence_after();
              scores(s, pos, 0);
              mma_commit(b_empty + 8 * (pos % NST));
              mma_commit(b_s + 8 * s);
              pos++;
            }
          }
        } else {
          const bool two = p.rows > 128;
          if (!(ok = full(pos))) break;
          tmem_fence_after();
          for (int s = 0; s < (two ? 2 : 1); s++) {
            scores(s, pos, s);
            mma_commit(b_s + 8 * s);
          }
          mma_commit(b_empty + 8 * (pos % NST));
          pos++;
          for (int t = 0; ok && t < n; t++) {
            const uint32_t pv = pos, pk = pos + 1;
            const bool more = t + 1 < n;
            if (!(ok = full(pv) && (!more || full(pk)))) break;
            for (int s = 0; s < (two ? 2 : 1); s++) {
              if (!(ok = weights(s))) break;
              tmem_fence_after();
              outputs(s, pv, t > 0);
              if (s == (two ? 1 : 0)) mma_commit(b_empty + 8 * (pv % NST));
              if (more) {
                scores(s, pk, s);
                if (s == (two ? 1 : 0)) mma_commit(b_empty + 8 * (pk % NST));
                mma_commit(b_s + 8 * s);
              }
            }
            pos += more ? 2 : 1;
          }
        }
        mma_commit(b_o);
      }
      // given up: what was issued ends before tensor memory is freed
      if (*abort) {
        mma_commit(b_drain);
        for (uint32_t i = 0; i < 1u << 16 && !bar_try(b_drain, 0); i++) {}
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- the walk
    if (lane == 0) {
      uint32_t at = 0;
      bool ok = true;
      auto hand = [&](const Piece& x) {
        // a piece may take long: this wait has the longer limit (10 s and more)
        ok = at < AT_PIECES;
        for (uint32_t i = 0; !ok && i < 1u << 26 && !*abort; i++) {
          ok = bar_try(b_taken + 8 * (at % AT_PIECES), (at / AT_PIECES + 1) & 1);
          if (!ok) __nanosleep(200);
        }
        if (!ok) {
          *abort = 1;
          return;
        }
        s_piece[at % AT_PIECES] = x;
        bar_arrive(b_piece + 8 * (at % AT_PIECES));
        at++;
      };
      Piece x = {};
      const int64_t end = min(total, x0 + share);
      int64_t u = x0 < total ? s_walk[1] : end;  // where a request, then a unit starts
      for (int64_t r = x0 < total ? s_walk[0] : a.R; ok && u < end && r < a.R; r++) {
        const Request q = load_request<ROWS>(a, r);
        for (int m = 0; ok && u < end && m < q.tiles_m; m++) {
          const int keys = unit_keys<ROWS>(a, q, m), tiles = key_tiles(keys), cost = tiles + AT_UNIT_COST;
          if (u + (int64_t)cost * a.hk <= x0) {
            u += (int64_t)cost * a.hk;
            continue;
          }
          for (int h = 0; ok && u < end && h < a.hk; h++, u += cost) {
            const int64_t t = u + AT_UNIT_COST;  // tile 0
            const int lo = (int)max((int64_t)0, min((int64_t)tiles, x0 - t)), hi = (int)min((int64_t)tiles, end - t);
            if (hi <= lo) continue;
            x.t0 = (int)q.t0;
            x.r = (int)r;
            x.h = h;
            x.row0 = m * ROWS;
            x.rows = min(ROWS, q.n * a.group - x.row0);
            x.n = q.n;
            x.ctx = q.ctx;
            x.len = q.len;
            x.open = !q.good ? 0 : a.mask ? q.ctx : q.ctx + x.row0 / a.group + 1;
            x.keys = keys;
            x.lo = lo;
            x.hi = hi;
            x.first = (int)(t / share);
            x.pieces = (int)((t + tiles - 1) / share) - x.first + 1;
            x.valid = 1 + q.good;
            hand(x);
          }
        }
      }
      x.valid = 0;
      hand(x);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ---- softmax: a thread has one row
    const int stream = (warp - 4) >> 2, wq = warp & 3, row = wq * 32 + lane, sid = tid - 128;
    const uint32_t t_lane = (uint32_t)(wq * 32) << 16;
    const uint32_t t_s = tmem + t_lane + stream * 128, t_o = tmem + t_lane + 256;
    const float c = a.scale_log2;
    uint32_t ns = 0, ring = 0, units = 0;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {  // one answer for the warp
      return __all_sync(0xffffffffu, bar_wait(bar, parity, abort)) != 0;
    };
    while (ok && __all_sync(0xffffffffu, next())) {
      __syncwarp();
      if (lane == 0) release();
      else taken++;
      const int n = p.hi - p.lo, rows = p.rows, row0 = p.row0, open = p.open;
      // queries into 128-byte swizzled rows
      {
        const T* q = static_cast<const T*>(a.q);
        for (int i = sid; i < rows * (D / 8); i += 256) {
          const int rr = i / (D / 8), ch = i % (D / 8);
          const int gr = row0 + rr, tok = gr / a.group;
          const uint4 x = *reinterpret_cast<const uint4*>(q + (p.t0 + tok) * a.q_stride +
                                                          (p.h * a.group + (gr - tok * a.group)) * D + ch * 8);
          const int tile = rr >> 7, r7 = rr & 127;
          *reinterpret_cast<uint4*>(smem + tile * (128 * D * 2) + (ch >> 3) * (128 * 128) + r7 * 128 + (((ch & 7) ^ (r7 & 7)) << 4)) = x;
        }
        fence_async_smem();
        tmem_fence_before();  // the last unit's output has been read
        bar_arrive(b_q);
      }
      const int my = (TILES == 2 ? stream * 128 : 0) + row;
      const bool live = my < rows;
      const bool active = (TILES == 2 ? stream * 128 : 0) + wq * 32 < rows;  // of the warp
      const int gr = row0 + my, tok = live ? gr / a.group : 0;
      Seen seen;
      seen.tree = a.mask != nullptr;
      seen.ctx = p.ctx;
      seen.last = p.valid == 2 ? p.ctx + tok : -1;
      seen.mask = 0;
      if (seen.tree && live && p.valid == 2) {
        seen.mask = (uint64_t)a.mask[p.t0 + tok];
        if (p.n < 64) seen.mask &= (1ull << p.n) - 1;
      }
      float m = -INFINITY, l = 0.f;
      const bool idle = TILES == 2 && stream * 128 >= rows;  // no second row tile

      for (int t = TILES == 1 ? stream : 0; !idle && t < n; t += TILES == 1 ? 2 : 1) {
        const int k0 = (p.lo + t) * AT_KEYS;
        const bool masked = k0 + AT_KEYS > open;
        if (!(ok = wait(b_s + 8 * stream, ns++ & 1))) break;
        tmem_fence_after();
        if (active) {
          uint32_t s[128];
#pragma unroll
          for (int i = 0; i < 4; i++) tmem_ld32(s + 32 * i, t_s + 32 * i);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const uint32_t w = seen.bits(k0 + 32 * i);
#pragma unroll
              for (int e = 0; e < 32; e++)
                if (!((w >> e) & 1)) s[32 * i + e] = 0xff800000u;
            }
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 128; i++) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(s[i]));
          const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          const bool first = t < (TILES == 1 ? 2 : 1);  // the stream's first tile
          const bool grow = live && mx > m && !((mx - m) * c <= 8.f);
          if (!first && __any_sync(0xffffffffu, grow)) {
            // the products before S are done: O is ours
            const float f = grow ? exp2_fast((m - mx) * c) : 1.f;
#pragma unroll
            for (int i = 0; i < D / 32; i++) {
              uint32_t o[32];
              tmem_ld32(o, t_o + stream * 128 + 32 * i);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(t_o + stream * 128 + 32 * i, o);
            }
            l *= f;
          }
          if (first || grow) m = mx;
          const float mc = m == -INFINITY ? 0.f : m * c;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 2; i++) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; e++) {
              const float p0 = exp2_fast(fmaf(__uint_as_float(s[64 * i + 2 * e]), c, -mc));
              const float p1 = exp2_fast(fmaf(__uint_as_float(s[64 * i + 2 * e + 1]), c, -mc));
              sum[(2 * e) & 3] += p0;
              sum[(2 * e + 1) & 3] += p1;
              w[e] = pack2<T>(p0, p1);
            }
            tmem_st32(t_s + 32 * i, w);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        if (masked && (TILES == 1 || stream == 0)) {
          // Values of keys past the request's end become 0; so do infinities and NaN of
          // keys that only some rows see: 0 * inf in a product would reach the others.
          // (rows that do see them get them back below)
          const uint32_t at = ring + (TILES == 2 ? 2 * t + 1 : n < 2 ? 1 : t == n - 1 ? 2 * n - 1 : 2 + 2 * t);
          if (!(ok = wait(b_full + 8 * (at % NST), (at / NST) & 1))) break;
          const int key = k0 + row;
          if (key >= open) {
            uint8_t* v = smem + L::Q + (at % NST) * L::STAGE + row * 128;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < D / 8; i++) {
              uint4* x = reinterpret_cast<uint4*>(v + (i >> 3) * (AT_KEYS * 128) + (((i & 7) ^ (row & 7)) << 4));
              if (key >= p.len) {
                *x = make_uint4(0, 0, 0, 0);
              } else {
                uint4 y = *x;
                uint32_t* z = reinterpret_cast<uint32_t*>(&y);
                const uint32_t any = nonfinite2<T>(z[0]) | nonfinite2<T>(z[1]) | nonfinite2<T>(z[2]) | nonfinite2<T>(z[3]);
                if (any) {
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
            if (bad) s_bad[units & 1] = 1;
          }
          fence_async_smem();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(b_p + 8 * stream);
      }
      ring += 2 * n;
      if (!ok || !(ok = wait(b_o, units & 1))) break;
      tmem_fence_after();
      if (sid == 0) s_bad[(units + 1) & 1] = 0;  // read by all in the unit before, written from the next on

      const bool whole = p.pieces == 1;
      float f0 = 1.f, f1 = 0.f;
      int d0 = 0, d1 = D;
      if (TILES == 1) {
        // both streams' rows: 2^(c m) l each, O in their own columns; a stream writes half of the columns
        s_ml[stream * 128 + row] = make_float2(m, l);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float2 x = s_ml[row], y = s_ml[128 + row];
        m = fmaxf(x.x, y.x);
        f0 = x.x == -INFINITY ? (x.y == 0.f ? 0.f : 1.f) : exp2_fast((x.x - m) * c);
        f1 = y.x == -INFINITY ? (y.y == 0.f ? 0.f : 1.f) : exp2_fast((y.x - m) * c);
        l = x.y * f0 + (n > 1 ? y.y * f1 : 0.f);
        d0 = stream * (D / 2);
        d1 = d0 + D / 2;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse2 = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * c) + log2f(l);
      const bool bad = s_bad[units & 1] != 0;
      float* part = part_at<D, ROWS>(a, blockIdx.x, p.lo == 0);
      const int64_t o_at = (int64_t)(p.t0 + tok) * a.hq + p.h * a.group + (gr - tok * a.group);
      if (active && !idle) {
        for (int d = d0; d < d1; d += 32) {
          uint32_t x[32];
          tmem_ld32(x, t_o + (TILES == 2 ? stream * 128 : 0) + d);
          tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; e++) o[e] = l == 0.f ? 0.f : __uint_as_float(x[e]) * f0;
          if (TILES == 1 && n > 1) {
            tmem_ld32(x, t_o + 128 + d);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = l == 0.f ? 0.f : fmaf(__uint_as_float(x[e]), f1, o[e]);
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] *= inv;
            if (bad) {
              // the values taken out above, for the rows that see them: any weight makes them infinite or NaN
              const int from = max(open, p.lo * AT_KEYS), to = min(p.len, p.hi * AT_KEYS);
              for (int j = from; j < to; j++) {
                if (!seen.has(j)) continue;
                const int64_t id = a.table[(int64_t)p.r * a.table_stride + (j >> a.log2_bs)];
                if (id < 0 || id >= a.n_blocks) continue;
                const T* v = reinterpret_cast<const T*>(a.v) + id * a.s_block + p.h * a.s_head +
                             (j & ((1 << a.log2_bs) - 1)) * a.s_token + d;
#pragma unroll
                for (int e = 0; e < 32; e++) {
                  const float y = (float)v[e];
                  if (!(fabsf(y) < INFINITY)) o[e] += y;
                }
              }
            }
            if (whole) {
              T* dst = static_cast<T*>(a.out) + o_at * D + d;
#pragma unroll
              for (int e = 0; e < 4; e++)
                *reinterpret_cast<uint4*>(dst + 8 * e) = make_uint4(pack2<T>(o[8 * e], o[8 * e + 1]), pack2<T>(o[8 * e + 2], o[8 * e + 3]),
                                                                    pack2<T>(o[8 * e + 4], o[8 * e + 5]), pack2<T>(o[8 * e + 6], o[8 * e + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(part + (int64_t)my * D + d);
#pragma unroll
              for (int e = 0; e < 8; e++) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
          __syncwarp();
        }
        if (live && (TILES == 2 || stream == 0)) {
          if (!whole) part[ROWS * D + my] = lse2;
          else if (a.lse) a.lse[o_at] = lse2 * 0.69314718055994531f;
        }
      }
      if (!whole) {
        // the CTA that finishes a divided unit last joins its pieces, always in their order on the line
        __threadfence();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const int np = p.pieces, first = p.first;
        if (sid == 0) {
          const unsigned done = atomicAdd(a.counters + first, 1u);
          *s_last = done == (unsigned)np - 1;
          if (done == (unsigned)np - 1) a.counters[first] = 0;
          __threadfence();
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (*s_last) {
          for (int i = sid; i < rows * (D / 4); i += 256) {
            const int rr = i / (D / 4), ch = i % (D / 4);
            float top = -INFINITY;
            for (int k = 0; k < np; k++) top = fmaxf(top, __ldcg(part_at<D, ROWS>(a, first + k, k == 0) + ROWS * D + rr));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float w = 0.f;
            for (int k = 0; k < np; k++) {
              const float* src = part_at<D, ROWS>(a, first + k, k == 0);
              const float e = __ldcg(src + ROWS * D + rr);
              const float4 x = __ldcg(reinterpret_cast<const float4*>(src + (int64_t)rr * D) + ch);
              if (e == -INFINITY) continue;
              const float f = exp2_fast(e - top);
              w += f;
              o.x = fmaf(f, x.x, o.x);
              o.y = fmaf(f, x.y, o.y);
              o.z = fmaf(f, x.z, o.z);
              o.w = fmaf(f, x.w, o.w);
            }
            const float wi = w == 0.f ? 0.f : 1.f / w;
            const int g = row0 + rr, tk = g / a.group;
            const int64_t to = (int64_t)(p.t0 + tk) * a.hq + p.h * a.group + (g - tk * a.group);
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + to * D + ch * 4) =
                make_uint2(pack2<T>(o.x * wi, o.y * wi), pack2<T>(o.z * wi, o.w * wi));
            if (a.lse && ch == 0) a.lse[to] = w == 0.f ? -INFINITY : (top + log2f(w)) * 0.69314718055994531f;
          }
        }
      }
      units++;
    }
  }
  if (*abort && lane == 0 && atomicCAS(&a.status->code, 0, TK_E_TIMEOUT) == 0) a.status->request = -1;
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    tmem_free(tmem);
  }
}

template <class T, int D, int TILES>
static cudaError_t attend_launch(const AttendArgs& a, const tk_kv_cache* cache, int grid, cudaStream_t st) {
  constexpr int bytes = AttendSmem<D, TILES>::TOTAL;
  static bool set[64];  // by device
  if (cache->device >= 64 || !set[cache->device]) {
    const cudaError_t e = cudaFuncSetAttribute(k_kv_attend<T, D, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (cache->device < 64) set[cache->device] = true;
  }
  k_kv_attend<T, D, TILES><<<grid, AT_THREADS, bytes, st>>>(a, cache->map_k, cache->map_v);
  return cudaGetLastError();
}

template <class T>
static cudaError_t attend_pick(const AttendArgs& a, const tk_kv_cache* cache, bool two, int grid, cudaStream_t st) {
  if (cache->head_dim == 64)
    return two ? attend_launch<T, 64, 2>(a, cache, grid, st) : attend_launch<T, 64, 1>(a, cache, grid, st);
  return two ? attend_launch<T, 128, 2>(a, cache, grid, st) : attend_launch<T, 128, 1>(a, cache, grid, st);
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
  // one block: the partial outputs of two pieces of every CTA, its counter, the status
  const size_t part = sizeof(float) * 2 * 256 * (128 + 1) * (size_t)ws->sms, counters = sizeof(unsigned) * (size_t)ws->sms;
  uint8_t* mem = nullptr;
  if (e == cudaSuccess) e = cudaMalloc(&mem, part + counters + 64 + sizeof(KvStatus));
  if (e == cudaSuccess) {
    ws->part = reinterpret_cast<float*>(mem);
    ws->counters = reinterpret_cast<unsigned*>(mem + part);
    ws->status = reinterpret_cast<KvStatus*>(mem + (part + counters + 63) / 64 * 64);
    e = cudaMemset(ws->counters, 0, counters + 64 + sizeof(KvStatus));
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
  KvStatus s = {};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  cudaError_t e = cudaMemcpyAsync(&s, ws->status, sizeof(s), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && s.code) e = cudaMemsetAsync(ws->status, 0, sizeof(s), st);
  // a call that gave up may have left counts behind
  if (e == cudaSuccess && s.code == TK_E_TIMEOUT) e = cudaMemsetAsync(ws->counters, 0, sizeof(unsigned) * ws->sms, st);
  if (e != cudaSuccess) {
    tk_set_error("tk_kv_status: %s", cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  if (s.code) {
    if (h_request) *h_request = s.request;
    if (s.code == TK_E_TIMEOUT) tk_set_error("tk_kv_attend: a wait on the device gave up");
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
  if (R < 0 || T < 0 || R > INT32_MAX || T > 1 << 26 || max_new < 0 || table_width < 0 || table_stride < table_width)
    return attend_arg(where, "bad size");
  if (q_stride < (int64_t)n_q_heads * cache->head_dim || q_stride % 8)
    return attend_arg(where, "q_stride is below a token's elements or no multiple of 8");
  if (!(scale > 0.f) || scale > 3e38f) return attend_arg(where, "scale is not a positive number");
  if (T * (n_q_heads / cache->n_heads) > INT32_MAX) return attend_arg(where, "T times the heads of a group is above 2^31");
  if (T == 0 || R == 0) return TK_OK;
  if (!d_q || !d_off || !d_len || !d_out || (table_width > 0 && !d_table)) return attend_arg(where, "null pointer");
  if ((((uintptr_t)d_q | (uintptr_t)d_out) & 15) != 0) return attend_arg(where, "a buffer is not 16-byte aligned");
  // a request's rows for one key head fill one row tile, or two and more
  const int group = n_q_heads / cache->n_heads;
  const bool two = std::min(max_new, T) * group > 128;
  AttendArgs a = {d_q, q_stride, n_q_heads, cache->n_heads, group, d_off, R, T, max_new, d_len, d_table, table_stride,
                  table_width, d_mask, scale * 1.4426950408889634f, d_out, d_lse, ws->status,
                  static_cast<const uint8_t*>(cache->v), cache->n_blocks, cache->stride[0], cache->stride[1],
                  cache->stride[2], cache->log2_block, ws->part, ws->counters};
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const cudaError_t e = cache->type == TK_BF16 ? attend_pick<__nv_bfloat16>(a, cache, two, ws->sms, st)
                                               : attend_pick<__half>(a, cache, two, ws->sms, st);
  if (e != cudaSuccess) {
    tk_set_error("%s: %s", where, cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  return TK_OK;
}
