// tk_attend_mma.cuh -- attention of new and drafted tokens over the paged cache
// (tk_kv_attend, tk_kv_attend_window) with the 5th-generation tensor cores: o = sum_j softmax_j(scale q.k_j) v_j over the keys j that a
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
// first accesses (200 keys: 12 us).  With a window: HBM for single tokens (64 requests, 4,096 of 14k
// each: 180 us, 6.0 TB/s), for prompts the starts and masked tiles of short units (2,000 tokens
// of 4 requests with a window of 1,024: 241 us, 0.61 PFLOP/s; with 4,096 1.10; without one 1.32).
// Over a cache in 8 bits 17 to 128 rows are bound by shared memory: for 64 keys of head_dim 128 a stream
// has 16 KB written by TMA, read again, 32 KB written as fp16, and 64 KB read by the products, which is 76% of what two streams'
// time has room for (eight tokens of 64 requests over 6k: 268 us; without turning the tiles 232).  More rows as above:
// 64 drafted tokens over 131k 247 us, without the exponentials 231.  (Both without a part when the whole took 270 and 256:
// weights were relative to the scales' largest.)
#pragma once
#include <type_traits>

#include "tk_attend.cuh"

namespace tk {

// A CTA: loads and products of two streams (4 warps), their softmax (2 x 4 warps); E8: 4 warps more.
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
constexpr int AT_PIECES = 4;  // handed over ahead

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
//
// E8: a cache in 8 bits.  Its tiles arrive as they are; four more warps turn them into fp16 for the products, which
// e4m3 is a subset of, so nothing is lost; queries of bf16 become fp16 with a power of two for each row (see
// tk_attend8.cu, which has the mathematics and takes calls of few rows).  The scales stay outside: a
// group of 16 keys lies in one block, its keys' scale is a factor of the group's scores, the log2 of its values' scale a summand
// of the weights' exponents; m is the bound M there, bound the bound R.
template <int D, int MODE, bool E8 = false>
struct AttendShape {
  static constexpr int THREADS = E8 ? 512 : 384;
  // E8, registers of a thread: 512 x 128 at launch = 128 x REGS_LOAD + 128 x REGS_TURN + 256 x REGS_SOFTMAX.  Eight tokens of
  // 64 requests over 6k, 64 rows a key head: 276 us with 88, 88 and 168, 272 so; MODE 2 with 184 for the softmax loses 5%.
  static constexpr int REGS_LOAD = MODE == 2 ? 80 : 112, REGS_TURN = MODE == 2 ? 48 : 64, REGS_SOFTMAX = MODE == 2 ? 192 : 168;
  static_assert(REGS_LOAD + REGS_TURN + 2 * REGS_SOFTMAX == 4 * 128, "no more than the CTA has");
  static constexpr int RINGS = MODE == 2 ? 1 : 2, ROWS = MODE == 0 ? 32 : MODE == 1 ? 128 : 256;
  static constexpr int Q_ROWS = MODE == 0 ? 32 : 128;  // of a stream
  static constexpr int KEYS = MODE == 2 ? 128 : 64, BUFS = 128 / KEYS;  // keys of a tile; tiles' scores in tensor memory
  // Up to 128 rows memory is the bound, which fewer workers reach too, so a worker with a single piece may have a
  // quarter more: 32 trees of 16 over 8k, 256 units for 304 workers, take 159 us padded (128 tiles each) and 189 us
  // divided evenly (108), 30 trees of 8 over 3k 62 and 77, one token of 32 requests over 8k of head_dim 64 109 and
  // 106.  The 8 tiles are for more rows: two trees of 64 over 30k take 67 us padded and 82 us not.
  template <bool WIN>
  using Tiles = Tiling<ROWS, KEYS, 1, WIN, AT_UNIT_COST, AT_MIN_SHARE, AT_SNAP, 8, MODE != 2>;
  static constexpr int Q = Q_ROWS * D * 2, STAGE = KEYS * D * 2;
  static constexpr int RING_BYTES = (RINGS == 1 ? 160 : MODE == 0 ? 96 : 80) * 1024;
  // of a ring; E8: three fifths of it hold fp16, the rest what arrives
  static constexpr int STAGES = (E8 ? RING_BYTES * 3 / 5 : RING_BYTES) / STAGE;
  static constexpr int RAW = STAGE / 2, RAWS = E8 ? RING_BYTES * 2 / 5 / RAW : 0;
  static constexpr int RING = 2 * Q;
  // barriers: full and empty of the stages; pieces handed over and taken; per stream q, s (2), p (2), v, o ready, o free, drain,
  // turn
  static constexpr int RAW_RING = RING + RINGS * STAGES * STAGE;
  static constexpr int BARS = RAW_RING + RINGS * RAWS * RAW;
  static constexpr int N_BARS = RINGS * (2 * STAGES + 2 * AT_PIECES) + 2 * 10 + RINGS * 2 * RAWS;  // and full and empty of the raw stages
  static constexpr int RAW_BARS = BARS + 8 * (RINGS * (2 * STAGES + 2 * AT_PIECES) + 2 * 10);
  static constexpr int PIECES = BARS + 8 * N_BARS;
  // scales of a tile's groups, keys' and log2 of values'; more tiles than are on their way
  static constexpr int GROUPS = KEYS / 16, SCALED = 16;
  static constexpr int SCALES = PIECES + RINGS * AT_PIECES * (int)sizeof(Piece);
  static constexpr int SMALL = SCALES + (E8 ? RINGS * SCALED * GROUPS * 8 : 0);
  static_assert(!E8 || STAGES + RAWS < 2 * SCALED, "a tile's scales are read before the next ones take their place");
  // start of the walk (2 x 2), sums, units and longest of the warps, tensor memory, abort, non-finite values (2 x 8)
  static constexpr int TOTAL = SMALL + 16 + 16 * (THREADS / 32) + 72;
  static_assert(STAGES >= 3 && SMALL % 8 == 0 && TOTAL <= 227 * 1024, "shared memory of one CTA");
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
//
// WIN: the call has a window.  A unit then reads the tiles of the first places and those from its first
// token's window on; a tile that only some of its rows see all of is masked, its values made finite,
// like one at the unit's end.
template <class T, int D, int MODE, bool LSE, bool WIN, bool E8>
__global__ void __launch_bounds__(E8 ? 512 : 384, 1)
k_kv_attend(const AttendArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using L = AttendShape<D, MODE, E8>;
  using H = std::conditional_t<E8, __half, T>;  // of the products
  constexpr int AT_THREADS = L::THREADS;
  constexpr int KEYS = L::KEYS, BUFS = L::BUFS, HALVES = D / 64, NST = L::STAGES;
  using S = typename L::template Tiles<WIN>;
  constexpr bool BF = Pair<H>::BF;
  // fp16 weights have their range below 2^15: with m's weight at 2^7 those 2^8 above it (before O is
  // rescaled) still fit, and one is lost at 2^-32 of m's instead of 2^-25: a million keys that
  // are each just below come to half an ulp of one of m's weight.
  constexpr float UP = BF ? 0.f : 7.f;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle goes by address bits
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stream = warp < 4 ? (warp >> 1) : warp < 12 ? (warp - 4) >> 2 : (warp - 12) >> 1;  // warps 0, 1 | 2, 3
  const int ring = MODE == 2 ? 0 : stream;
  const uint32_t s_ring = base + L::RING + ring * (NST * L::STAGE), s_q = base + stream * L::Q;
  const uint32_t b_full = base + L::BARS + ring * 8 * (2 * NST + 2 * AT_PIECES), b_empty = b_full + 8 * NST,
                 b_piece = b_empty + 8 * NST, b_taken = b_piece + 8 * AT_PIECES;
  const uint32_t b_q = base + L::BARS + L::RINGS * 8 * (2 * NST + 2 * AT_PIECES) + stream * 80, b_s = b_q + 8, b_p = b_s + 16,
                 b_v = b_p + 16, b_o = b_v + 8, b_free = b_o + 8, b_drain = b_free + 8, b_turn = b_drain + 8;
  const uint32_t s_raw = base + L::RAW_RING + ring * (L::RAWS * L::RAW);
  const uint32_t b_raw = base + L::RAW_BARS + ring * 16 * L::RAWS, b_used = b_raw + 8 * L::RAWS;
  float2* s_scale = reinterpret_cast<float2*>(smem + L::SCALES) + ring * (L::SCALED * L::GROUPS);
  Piece* s_piece = reinterpret_cast<Piece*>(smem + L::PIECES) + ring * AT_PIECES;
  int* s_walk = reinterpret_cast<int*>(smem + L::SMALL);  // of each worker: first request, where it starts
  int* s_sum = s_walk + 4;
  volatile int* s_int = reinterpret_cast<volatile int*>(s_sum + 4 * AT_THREADS / 32);
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
      constexpr int TURNING = E8 ? (MODE == 2 ? 4 : 2) : 0;  // warps of a ring that turn its tiles into fp16
      if (st < 0) {
        if (E8 && in < NST) count = TURNING;
        else if (in >= NST && in < 2 * NST) count = MODE == 2 ? 2 : 1;           // empty: the streams that read the stage
        else if (in >= 2 * NST + AT_PIECES) count = (MODE == 2 ? 10 : 5) + TURNING;  // taken: products and softmax warps
      } else if (st >= 20) {
        if ((st - 20) % (2 * L::RAWS + (L::RAWS == 0)) >= L::RAWS) count = TURNING;
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
  constexpr int WORKERS = MODE == 2 ? 1 : 2;  // of a CTA
  Plan plan;
  const int total = make_plan<S, AT_THREADS, WORKERS, D>(a, plan, s_sum, s_walk);
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

  // registers: 384 x 168 at launch = 128 x 104 + 256 x 200, where a softmax thread holds 128 scores;
  // E8: see AttendShape
  if (warp < 4) {
    if (E8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::REGS_LOAD));
    else if (MODE == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0 || (warp == 3 && MODE != 2)) {
      // ---- loads, in the order of their use: K0 K1 V0 K2 V1 K3 ... with two tiles' scores, K0 V0 K1 V1 ... with one
      Walk<S> walk;
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
      // (E8: of all elements)
      const int log2_box = min(a.log2_bs, 6), per_page = a.log2_bs - log2_box, ppt = KEYS >> log2_box;
      const int my_box = E8 ? lane : lane / HALVES, my_half = E8 ? 0 : lane % HALVES;
      const uint32_t my_dst = E8 ? s_raw + (my_box * D << log2_box) : s_ring + my_half * (KEYS * 128) + (my_box * 128 << log2_box);
      const uint32_t box_bytes = E8 ? (uint32_t)D << log2_box : HALVES * 128u << log2_box;
      constexpr int NLD = E8 ? L::RAWS : NST, LD = E8 ? L::RAW : L::STAGE;  // the stages that are loaded
      const uint32_t b_land = E8 ? b_raw : b_full, b_left = E8 ? b_used : b_empty;
      uint32_t scaled = 0;  // tiles whose scales have been handed over
      // block ids: a lane has box `window + lane`, and the one 32 further on
      // (and of keys the scales of the former)
      struct Ids {
        int window, now, then;
        float2 scale;
      };
      int boxes = 0, h = 0, head = 0, skip = 0;
      const int32_t* row = nullptr;
      auto at_key = [&](int tile) { return WIN && tile >= head ? tile + skip : tile; };  // in tiles from key 0 on
      auto id_of = [&](int b) { return b < boxes ? __ldg(row + (b >> per_page)) : 0; };
      auto scale_of = [&](int id) {
        if (id < 0 || id >= a.n_blocks) return make_float2(0.f, E8_NONE);
        const int64_t at = (int64_t)id * a.hk + h;
        return make_float2(__ldg(a.k_scale + at), e8_log2(__ldg(a.v_scale + at)));
      };
      auto load = [&](const CUtensorMap* map, Ids& ids, int tile, bool keys) {
        const int box0 = at_key(tile) * ppt;
        if (box0 >= ids.window + 32) {
          if (WIN && box0 >= ids.window + 64) {
            ids.window = box0 & ~31;
            ids.now = id_of(ids.window + lane);
          } else {
            ids.window += 32;
            ids.now = ids.then;
          }
          ids.then = id_of(ids.window + 32 + lane);
          if (E8 && keys) ids.scale = scale_of(ids.now);
        }
        const int nb = max(0, min(ppt, boxes - box0));
        const int id = __shfl_sync(0xffffffffu, ids.now, (box0 + my_box) & 31);
        if (E8 && keys) {
          const int of = lane >> (log2_box - 4);  // the box of group `lane`
          const float ks = __shfl_sync(0xffffffffu, ids.scale.x, (box0 + of) & 31), vs = __shfl_sync(0xffffffffu, ids.scale.y, (box0 + of) & 31);
          if (lane < L::GROUPS) s_scale[(scaled % L::SCALED) * L::GROUPS + lane] = of < nb ? make_float2(ks, vs) : make_float2(0.f, E8_NONE);
          scaled++;
          __syncwarp();
        }
        if (filled == NLD) {
          ok = __all_sync(0xffffffffu, bar_wait(b_left + 8 * st, ph ^ 1, abort)) != 0;
          if (!ok) return;
        } else {
          filled++;
        }
        if (elect_one()) bar_expect(b_land + 8 * st, nb * box_bytes);
        __syncwarp();
        if (my_box < nb)
          tma_load_4d(my_dst + st * LD, map, b_land + 8 * st, my_half * 64, ((box0 + my_box) & ((1 << per_page) - 1)) << log2_box, h, id);
        if (++st == NLD) st = 0, ph ^= 1;
      };
      walk.seek(a);
      Piece nx;
      walk.next(a, nx);
      hand(nx);
      while (ok && nx.valid) {
        const int lo = nx.lo, hi = nx.hi;
        h = nx.h;
        if (WIN) {
          head = nx.head;
          skip = nx.skip;
        }
        boxes = (nx.keys + (1 << log2_box) - 1) >> log2_box;
        row = a.table + (int64_t)nx.r * a.table_stride;
        Ids k, v;
        k.window = (at_key(lo) * ppt) & ~31;
        k.now = id_of(k.window + lane);
        k.then = id_of(k.window + 32 + lane);
        if (E8) k.scale = scale_of(k.now);
        v = k;
        for (int t = lo; ok && t < min(hi, lo + BUFS); t++) load(&map_k, k, t, true);
        for (int t = lo; ok && t < hi; t++) {
          load(&map_v, v, t, false);
          // the next piece is known to the softmax, which asks for it in its last tile, before
          // more loads wait for it
          if (ok && t == lo) {
            walk.next(a, nx);
            hand(nx);
          }
          if (ok && t + BUFS < hi) load(&map_k, k, t + BUFS, true);
        }
      }
      // given up: the copies in flight land before the CTA ends
      if (*abort)
        for (uint32_t k = 0; k < filled; k++) {
          const uint32_t x = st + NLD - filled + k;  // the stages filled last, oldest first
          for (uint32_t i = 0; i < 1u << 16 && !bar_try(b_land + 8 * (x % NLD), x >= NLD ? ph : ph ^ 1); i++) {}
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
          // (E8: these keys may be turned into fp16 only where the last tile's values were)
          if (more) {
            if (!E8 && !(ok = full())) break;
            if (!E8) advance();
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
            if (!E8 && more) scores(buf, sk);
            if (turn && !(E8 && more)) bar_arrive(b_turn);
          }
          __syncwarp();
          if (E8 && more) {
            if (!(ok = full())) break;
            advance();
            tmem_fence_after();
            if (elect_one()) {
              scores(buf, sk);
              if (turn) bar_arrive(b_turn);
            }
            __syncwarp();
          }
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
  } else if (E8 && warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::REGS_TURN));
    // ---- 8 bits to fp16, stage by stage.  A thread has 16 elements of a key at a time, the lanes of a
    // quarter-warp eight keys that follow one another: neither side meets a bank twice.
    constexpr int WARPS = MODE == 2 ? 4 : 2, CHUNKS = D / 16;
    const int me = (MODE == 2 ? tid - 384 : (tid - 384) & 63);
    uint32_t st = 0, ph = 0, rs = 0, rph = 0, filled = 0;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(bar, parity, abort)) != 0; };
    while (ok && coming(taken)) {
      const Piece& p = s_piece[taken % AT_PIECES];
      const int n = __shfl_sync(0xffffffffu, p.hi - p.lo, 0);
      release();
      for (int i = 0; i < 2 * n; i++) {
        if (!(ok = wait(b_raw + 8 * rs, rph))) break;
        if (filled == NST) {
          if (!(ok = wait(b_empty + 8 * st, ph ^ 1))) break;
        } else {
          filled++;
        }
        const uint32_t src = s_raw + rs * L::RAW, dst = s_ring + st * L::STAGE;
#pragma unroll 4
        for (int x = me; x < KEYS * CHUNKS; x += WARPS * 32) {
          const int key = x % KEYS, c = x / KEYS;
          uint32_t w[4], y[8];
          const uint32_t at = D == 128 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src + at));
#pragma unroll
          for (int e = 0; e < 4; e++) {
            y[2 * e] = e4m3_lo(w[e]);
            y[2 * e + 1] = e4m3_hi(w[e]);
          }
          const uint32_t to = dst + (c >> 2) * (KEYS * 128) + key * 128;
          const int c16 = (c & 3) * 2;
#pragma unroll
          for (int e = 0; e < 2; e++)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((c16 + e) ^ (key & 7)) << 4)), "r"(y[4 * e]),
                         "r"(y[4 * e + 1]), "r"(y[4 * e + 2]), "r"(y[4 * e + 3])
                         : "memory");
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(b_full + 8 * st);
          bar_arrive(b_used + 8 * rs);
        }
        if (++st == NST) st = 0, ph ^= 1;
        if (++rs == L::RAWS) rs = 0, rph ^= 1;
      }
    }
    __syncwarp();
  } else {
    if (E8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::REGS_SOFTMAX));
    else if (MODE == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax
    const int wq = warp & 3, row = wq * 32 + lane;  // row = also its lane of tensor memory
    const uint32_t t_s = ((uint32_t)(wq * 32) << 16) + stream * 256, t_o = t_s + 128;
    const float c = a.scale_log2;
    float qs = 1.f, qs_next = 1.f;  // E8: what the row's queries are to be multiplied by
    uint32_t scaled = 0;            // E8: tiles of pieces before this one
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
        const int rr = i / (D / 8), ch = i % (D / 8), gr = row0 + rr, tok = by_group(a, gr);
        const T* src = q + tok * a.q_stride + (gr - tok * a.group) * D + ch * 8;
        const uint32_t dst = s_q + (ch >> 3) * (L::Q_ROWS * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
      }
    };
    auto fetched = [&](uint32_t pc) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (E8 && Pair<T>::BF) {
        // bf16 to fp16, each thread its row: the largest element to 2^14
        stream_sync();
        if (row < s_piece[pc % AT_PIECES].rows - skip) {
          uint4* x = reinterpret_cast<uint4*>(smem + (s_q - base) + row * 128);
          auto chunk = [&](int i) -> uint4& { return x[(i >> 3) * (L::Q_ROWS * 8) + ((i & 7) ^ (row & 7))]; };
          uint32_t top = 0;
#pragma unroll 4
          for (int i = 0; i < D / 8; i++) {
            const uint4 y = chunk(i);
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const uint32_t w = reinterpret_cast<const uint32_t*>(&y)[e], lo = w & 0x7f80u, hi = (w >> 16) & 0x7f80u;
              if (lo < 0x7f80u) top = max(top, lo);
              if (hi < 0x7f80u) top = max(top, hi);
            }
          }
          const int e = min(max((int)(top >> 7), 40), 254);  // below 2^-87 nothing is left
          const float f = __uint_as_float((uint32_t)(268 - e) << 23);
          qs_next = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll 4
          for (int i = 0; i < D / 8; i++) {
            uint4 y = chunk(i);
#pragma unroll
            for (int k = 0; k < 4; k++) {
              uint32_t& w = reinterpret_cast<uint32_t*>(&y)[k];
              const float2 z = Pair<T>::up(*reinterpret_cast<const typename Pair<T>::type*>(&w));
              w = pack2<__half>(z.x * f, z.y * f);
            }
            chunk(i) = y;
          }
        }
      }
      fence_async_smem();
      bar_arrive(b_q);
    };
    auto has_rows = [&](uint32_t pc) { return MODE != 2 || s_piece[pc % AT_PIECES].rows > skip; };
    bool more = coming(0);
    if (more && has_rows(0)) {
      fetch(0);
      fetched(0);
    }
    while (more) {
      const Piece& p = s_piece[taken % AT_PIECES];  // released at the unit's end: registers are short
      const int n = p.hi - p.lo, rows = min(128, p.rows - skip), open = p.open;
      const uint32_t ring0 = stages;  // its first stage
      stages += 2 * n;
      const uint32_t scaled0 = scaled;  // its first tile
      scaled += n;
      qs = qs_next;
      if (rows <= 0) {  // nothing for this stream
        if ((more = coming(taken + 1)) && has_rows(taken + 1)) {
          fetch(taken + 1);
          fetched(taken + 1);
        }
        release();
        continue;
      }
      const bool live = row < rows, active = wq * 32 < rows;  // the row's, the warp's
      const int gr = p.row0 + skip + row, tok = live ? by_group(a, gr) : 0;
      Seen<WIN> seen;
      seen.set(a, p, live, tok);
      float m = E8 ? -E8_MOST : -INFINITY, l = 0.f, l_full = 0.f;
      float mc = 0.f;            // m c - UP, or 0 while the row has seen nothing
      float bound = -E8_MOST;    // E8
      const int lo = p.lo;
      const uint64_t c2 = pair64(c, c);

      // of the scores of a group; with the least normal number a hidden key's -infinity stays that
      const float cq = c * qs;
      auto factor = [&](float ks) { return fmaxf(cq * ks, 1.17549435e-38f); };
      const int head = p.head, jump = WIN ? p.skip : 0, shut = p.shut;
      auto at_key = [&](int tile) { return (WIN && tile >= head ? tile + jump : tile) * KEYS; };
      // a tile, a key
      auto seen_by_all = [&](int k0) { return k0 + KEYS <= open && (!WIN || k0 >= shut || k0 + KEYS <= a.sinks); };
      auto seen_by_some = [&](int key) { return key >= open || (WIN && key < shut && key >= a.sinks); };

      // One tile.  Nearly all are seen by every row; where the softmax is the bound (MODE 2) those have a
      // body of their own.
      auto tile = [&](int t, auto some_hidden) {
        const int k0 = at_key(lo + t);
        const bool hidden = decltype(some_hidden)::value && (MODE == 2 || !seen_by_all(k0));
        if (hidden) {
          // Values of keys past the unit's become 0 (what is not loaded there may be anything, and is no reason to
          // look for infinities below); so do infinities and NaN of
          // keys that only some rows see: 0 * inf in a product would reach the others.
          // (Rows that do see them get them back below.)  Streams that share a tile leave it to the first.
          if (MODE != 2 || stream == 0) {
            const uint32_t at = ring0 + (BUFS == 1 ? 2 * t + 1 : n == 1 ? 1 : t == n - 1 ? 2 * n - 1 : 2 * t + 2);
            // A wait tells one phase from the one before: the stage has to have been filled for its last tile, NST
            // stages ago. With three stages that is this tile's keys, which its scores are the sign of.
            if (NST < 4 && BUFS == 2) wait(b_s + 8 * (nt % BUFS), (nt / BUFS) & 1);
            wait(b_full + 8 * (at % NST), (at / NST) & 1);
            // 16 bytes a thread at a time, eight or sixteen keys a pass: those that every row sees are passed over
            constexpr int CHUNKS = D / 8;
            uint8_t* v = smem + (s_ring - base) + (at % NST) * L::STAGE;
            bool bad = false;
#pragma unroll 4
            for (int i = row; i < KEYS * CHUNKS; i += 128) {
              const int kr = i / CHUNKS, ch = i % CHUNKS, key = k0 + kr;
              if (!seen_by_some(key)) continue;
              uint4* x = reinterpret_cast<uint4*>(v + (ch >> 3) * (KEYS * 128) + kr * 128 + (((ch & 7) ^ (kr & 7)) << 4));
              // no row sees those past the unit's and before the first one's window
              if (key >= p.keys || (WIN && key >= a.sinks && key < open - a.window)) {
                *x = make_uint4(0, 0, 0, 0);
              } else {
                uint4 y = *x;
                uint32_t* z = reinterpret_cast<uint32_t*>(&y);
                if (nonfinite2<H>(z[0]) | nonfinite2<H>(z[1]) | nonfinite2<H>(z[2]) | nonfinite2<H>(z[3])) {
                  bad = true;
#pragma unroll
                  for (int e = 0; e < 4; e++) {
                    const uint32_t b = nonfinite2<H>(z[e]);
                    if (b & 0x8000u) z[e] &= 0xffff0000u;
                    if (b & 0x80000000u) z[e] &= 0x0000ffffu;
                  }
                  *x = y;
                }
              }
            }
            if (bad) s_bad[taken & 7] = 1;
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
          [[maybe_unused]] const float2* scales = s_scale + ((scaled0 + t) % L::SCALED) * L::GROUPS;
          float mx, my = -INFINITY;  // the largest score; E8: and with its value's scale
          if constexpr (E8) {
            mx = -INFINITY;
#pragma unroll
            for (int g = 0; g < L::GROUPS; g++) {
              float x = max3(__uint_as_float(s[16 * g]), __uint_as_float(s[16 * g + 1]), __uint_as_float(s[16 * g + 2]));
              float y = max3(__uint_as_float(s[16 * g + 3]), __uint_as_float(s[16 * g + 4]), __uint_as_float(s[16 * g + 5]));
#pragma unroll
              for (int i = 6; i < 14; i += 4) {
                x = max3(x, __uint_as_float(s[16 * g + i]), __uint_as_float(s[16 * g + i + 1]));
                y = max3(y, __uint_as_float(s[16 * g + i + 2]), __uint_as_float(s[16 * g + i + 3]));
              }
              x = max3(fmaxf(x, y), __uint_as_float(s[16 * g + 14]), __uint_as_float(s[16 * g + 15])) * factor(scales[g].x);
              mx = fmaxf(mx, x);
              my = fmaxf(my, x + scales[g].y);
            }
          } else {
            float top[4];
  #pragma unroll
            for (int i = 0; i < 4; i++) top[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
  #pragma unroll
            for (int i = 8; i < KEYS; i += 2)
              top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
            mx = fmaxf(max3(top[0], top[1], top[2]), top[3]);
          }
          // E8: of the sum another factor than of the output
          const bool grow = E8 ? live && my > bound : t == 0 || (live && mx > m && !((mx - m) * c <= 8.f));
          if (E8 && live && mx > m) {
            l *= exp2_fast(m - (mx + 8.f));
            m = mx + 8.f;
          }
          if (__any_sync(0xffffffffu, grow)) {
            if (t > 0) {
              // the products of the tile before may still run
              wait(b_v, (nt + 1) & 1);
              tmem_fence_after();
              const float f = !grow ? 1.f : E8 ? exp2_fast(bound - (my + 8.f)) : exp2_fast((m - mx) * c);
#pragma unroll 1
              for (int i = 0; i < D / 32; i++) {
                uint32_t o[32];
                tmem_ld32(o, t_o + 32 * i);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(t_o + 32 * i, o);
              }
              if (!E8) {
                l *= f;
                l_full *= f;
              }
            }
            if (grow) {
              if (E8) bound = my + 8.f;
              else {
                m = mx;
                mc = m == -INFINITY ? 0.f : fmaf(m, c, -UP);
              }
            }
          }
          const uint64_t mc2 = pair64(-mc, -mc);
          if constexpr (E8) {
            // a group's part of the sum is 2^-d times that of its weights
            float all[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < KEYS / 64; i++) {
              uint32_t w[32];
#pragma unroll
              for (int g = 0; g < 4; g++) {
                const float f = factor(scales[4 * i + g].x), d = e8_shift(scales[4 * i + g].y, m, bound);
                const uint64_t f2 = pair64(f, f), to = pair64(d - m, d - m);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int e = 8 * g; e < 8 * g + 8; e++) {
                  const float2 x = unpair64(fma2(pair64(s[64 * i + 2 * e], s[64 * i + 2 * e + 1]), f2, to));
                  const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y);
                  sum[e & 1] = add2(sum[e & 1], pair64(p0, p1));
                  w[e] = pack2<__half>(p0, p1);
                }
                const float2 sum2 = unpair64(add2(sum[0], sum[1]));
                all[g & 1] = fmaf(sum2.x + sum2.y, exp2_fast(-d), all[g & 1]);
              }
              tmem_st32(t_s + buf * KEYS + 32 * i, w);
            }
            l += all[0] + all[1];
          } else {
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
                w[e] = pack2<H>(p0, p1);
                add_halves(sum[2 * (e & 1)], sum[2 * (e & 1) + 1], w[e], BF);
              }
              tmem_st32(t_s + buf * KEYS + 32 * i, w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (LSE) {
              const float2 l2 = unpair64(add2(full[0], full[1]));
              l_full += l2.x + l2.y;
            }
          }
          tmem_wait_st();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(b_p + 8 * buf);
        nt++;
      };
      int clear = 0;
      if constexpr (MODE == 2 && !WIN) {
        clear = max(0, min(n, open / KEYS - lo));
#pragma unroll 1
        for (int t = 0; t < clear; t++) tile(t, std::false_type());
      }
#pragma unroll 1
      for (int t = clear; t < n; t++) {
        if (MODE == 2 && WIN && seen_by_all(at_key(lo + t))) tile(t, std::false_type());
        else tile(t, std::true_type());
      }
      // the queries have been read for the last time: the next ones come in under the last products
      more = coming(taken + 1);
      if (more && has_rows(taken + 1)) {
        fetch(taken + 1);
        fetched(taken + 1);
      }
      wait(b_o, units & 1);
      tmem_fence_after();

      const bool whole = p.pieces == 1;
      const bool bad = s_bad[taken & 7] != 0;
      float* part = part_at<D>(a.part, me, p.lo == 0);
      const int64_t o_at = (int64_t)(p.t0 + tok) * a.hq + p.h * a.group + (gr - tok * a.group);
      if (active) {
        // (E8: in two factors: of scales from 2^127 on it may be more than fp32 has)
        const float half = E8 ? exp2f(0.5f * (bound - E8_TOP - m)) : 1.f, inv = l == 0.f ? 0.f : half / l;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t x[32];
          tmem_ld32(x, t_o + d);
          tmem_wait_ld();
          if (live) {
            float o[32];
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = l == 0.f ? 0.f : E8 ? __uint_as_float(x[e]) * inv * half : __uint_as_float(x[e]) * inv;
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
            __stcg(part + 128 * D + row, l == 0.f ? -INFINITY : (E8 ? m : mc) + log2f(l));
            if (LSE) __stcg(part + 128 * D + 128 + row, l == 0.f || E8 ? 1.f : l_full / l);
          } else if (LSE && a.lse) {
            a.lse[o_at] = l == 0.f ? -INFINITY : ((E8 ? m : mc) + log2f(E8 ? l : l_full)) * 0.69314718055994531f;
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
        const int to = WIN ? n * KEYS : min(p.len, p.hi * KEYS);
        for (int i = WIN ? 0 : max(open, p.lo * KEYS); i < to; i++) {
          const int j = WIN ? at_key(lo + i / KEYS) + i % KEYS : i;
          if (WIN && (!seen_by_some(j) || j >= p.len)) continue;
          const int64_t id = a.table[(int64_t)p.r * a.table_stride + (j >> a.log2_bs)];
          if (!seen.has(j) || id < 0 || id >= a.n_blocks) continue;
          const int64_t v_at = id * a.s_block + p.h * a.s_head + (j & ((1 << a.log2_bs) - 1)) * a.s_token;
          for (int d = 0; d < D; d++) {
            float y;
            if (E8) y = (static_cast<const uint8_t*>(a.v)[v_at + d] & 0x7f) == 0x7f ? __int_as_float(0x7fffffff) : 0.f;
            else y = (float)static_cast<const T*>(a.v)[v_at + d];
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
          const int gr = join_g[k] + rr, tk = by_group(a, gr);
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

template <class T, int D, int MODE, bool LSE, bool WIN, bool E8>
static cudaError_t attend_launch(const AttendArgs& a, const tk_kv_cache* cache, int grid, cudaStream_t st) {
  constexpr int bytes = AttendShape<D, MODE, E8>::TOTAL;
  static bool set[64];  // by device
  if (cache->device >= 64 || !set[cache->device]) {
    const cudaError_t e = cudaFuncSetAttribute(k_kv_attend<T, D, MODE, LSE, WIN, E8>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (cache->device < 64) set[cache->device] = true;
  }
  cudaLaunchAttribute coop;
  coop.id = cudaLaunchAttributeCooperative;
  coop.val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(AttendShape<D, MODE, E8>::THREADS);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cfg.attrs = &coop;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv_attend<T, D, MODE, LSE, WIN, E8>, a, cache->map_k, cache->map_v);
}

// rows: of a request and key head, at most
template <class T, int D, bool WIN>
static cudaError_t attend_pick(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  if (rows <= 32) return attend_launch<T, D, 0, true, WIN, false>(a, cache, grid, st);
  if (rows <= 128) return attend_launch<T, D, 1, true, WIN, false>(a, cache, grid, st);
  // A window's units are short and begin and end with masked tiles: two streams of their own then do better than one pair.
  // Four prompts of 2,000 tokens, 275 instead of 298 us with a window of 1,024, 149
  // instead of 167 with 128, 553 instead of 584 with 4,096; 64 trees of 64 with 1,024 164 instead of 170.
  if constexpr (WIN) return attend_launch<T, D, 1, true, WIN, false>(a, cache, grid, st);
  else return a.lse ? attend_launch<T, D, 2, true, WIN, false>(a, cache, grid, st) : attend_launch<T, D, 2, false, WIN, false>(a, cache, grid, st);
}

template <bool WIN>
static cudaError_t attend_types(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  if (cache->type == TK_BF16)
    return cache->head_dim == 64 ? attend_pick<__nv_bfloat16, 64, WIN>(a, cache, rows, grid, st)
                                 : attend_pick<__nv_bfloat16, 128, WIN>(a, cache, rows, grid, st);
  return cache->head_dim == 64 ? attend_pick<__half, 64, WIN>(a, cache, rows, grid, st)
                               : attend_pick<__half, 128, WIN>(a, cache, rows, grid, st);
}

}  // namespace tk
