// tk_attend8.cu -- attention over a paged cache in 8 bits (tk_kv_attend, tk_kv_attend_window):
// o = sum_j softmax_j(scale ks_j q.k_j) vs_j v_j, k_j and v_j e4m3, ks_j and vs_j their block's scales.
//
// e4m3 is a subset of fp16, so keys and values enter the products exactly, as fp16, whatever the
// queries' type.  Queries of bf16 become fp16 with a power of two for each row that brings their largest element to
// 2^14: exact but for elements 2^-28 below it, which lose less than fp32's sums do.  The scales
// stay outside: the keys' is a factor of the scores (16 keys lie in one block), the
// values' of the weights.  Of each row
//   x_j = c ks_j (q.k_j), c = scale log2(e);  y_j = x_j + log2(vs_j);  l += 2^(x_j - M);
//   w_j = 2^(y_j - R + 15) rounded to fp16 (a choice: the products' other type, bf16, has 3 bits less), O += w_j v_j;
//   o = 2^(R - 15 - M) O / l.
// M and R are bounds of the x and the y that the row has seen: one that is passed is put 8 above what passed it, so that few
// steps pass it again; w is 2^7 at least of the row's largest y, and 2^15 at most.  What fp16 loses, its half step of 2^-25,
// is 2^-32 of the row's largest weight times scale and less: of both, so neither a block that the row
// does not see nor one of large scale and no weight takes anything from the others.
// l is summed from the same exponentials: with d = log2(vs) + M - R + 15, the same for a step's 16 keys, w = 2^(x - M + d)
// and its part of l is 2^-d of w.  d is kept from falling below -60, where nothing of w is left in fp16 and all of it in fp32;
// log2(vs) is finite whatever the scales of places that nobody sees are, so that these have the weight 0.
//
// The kernel here takes up to 16 rows (query heads of a key head x tokens), where memory is the bound by far, and the
// operands of tcgen05 would cost more shared memory traffic than the keys and values themselves (the two
// products of 64 keys of head_dim 128 read 64 KB, 512 cycles, and their tile in fp16 is another 64 KB written and
// read, where the 8-bit tile takes 700 cycles to arrive).  So a warp's products are those of its registers
// (m16n8k16), with keys and columns as their 16 and rows as their 8: S^T = K Q^T, O^T = V^T P^T.  It reads a
// key's 16 bytes as they are, four neighbouring elements being one thread's share of a product of 16, which may be any
// 16 as long as the queries take the same; of the values a thread has four keys' 16 bytes, whose bytes it pairs
// up.  Nothing is written to shared memory but what TMA brings.
// One token of 128 requests over 6k, 1.63 GB: 247 to 252 us, 6.5 TB/s, 96% of a copy's rate.  16 rows take 93 us for 400 MB
// (4.3 TB/s): the chain of a step's instructions, with three quarters of the warps for twice the rows' registers (of head_dim 128
// some are spilled: 148 to 268 bytes stored a thread, 80 to 88 loaded).  Of the way
// here, the same case: rows as the products' 16, 8 warps 337 us; steps of 32 keys 298; 12 warps 332; rows as
// their 8, 16 warps 267; a dearer unit 251; then weights relative to the largest scale of the values instead of
// to the row's bounds, which was wrong where scales are far apart, the same (16 rows 98).
// More rows go to the 5th-generation tensor cores (tk_attend8_mma.cu): 24 trees of up to 17 rows over 1.5k
// (head_dim 64) take 47 us there, and took 66 here with another 16 rows.
#include "tk_attend.cuh"

namespace tk {

constexpr int A8_STEP = 16;  // keys of a step, one warp's: they lie in one block

// NR: 8 rows each.  The work on 16 keys is a chain of instructions that wait for one another, so there are as many
// warps as their registers allow.  A warp has a ring of its own: STAGES steps of keys and values.
template <int D, int NR>
struct Attend8Shape {
  static constexpr int ROWS = 8 * NR, WARPS = NR == 1 ? 16 : 12, THREADS = WARPS * 32;
  static constexpr int TILE = A8_STEP * D, STAGE = 2 * TILE, STAGES = 8 * 1024 / STAGE;
  // outputs of the warps as they are joined, 8 rows at a time: [warp][8][O_ROW] floats, in which
  // the stores and loads of a quarter-warp meet no bank twice
  static constexpr int O_GROUP = D / 8 + 4, O_ROW = 8 * O_GROUP + 4;
  static constexpr int O = WARPS * STAGES * STAGE;
  static constexpr int STATS = O + WARPS * 8 * O_ROW * 4;  // [ROWS][warp] M, l, R
  static constexpr int BARS = STATS + 3 * ROWS * WARPS * 4;
  static constexpr int SMALL = BARS + 8 * WARPS * STAGES;
  static constexpr int PIECES = SMALL + 16 + 4 * WARPS * 4 + 16;  // this one and the next one; the walk
  static constexpr int TOTAL = PIECES + 2 * (int)sizeof(Piece) + 192;
  // What starting a unit costs, in tiles of a step for every warp; half of a worker's least share, and no cut is nearer to
  // a unit's ends.  Up to 8 rows, one token of 128 requests over 6k, of 64 over 1k and of 8 over 2k (us): 1: 269, 48, 19.2; 2:
  // 254, 46, 19.7; 3: 251, 45, 19.9; 4: 251, 44, 20.6; 6: 255, 47, 21.4.  Up to 16, one of 64 requests over 6k with 16 rows and
  // three with 12: 2: 106, 190; 4: 98, 176; 6: 97, 173; 8: 100, 174.  (Weights were relative to the scales' largest then; now 250,
  // 43, 19.5, and 93, 165.)
  static constexpr int UNIT_COST = NR == 1 ? 3 : 6;
  template <bool WIN>
  using Tiles = Tiling<ROWS, A8_STEP, WARPS, WIN, UNIT_COST, 2 * UNIT_COST, UNIT_COST, 2, true>;
  static_assert(SMALL % 8 == 0 && PIECES % 8 == 0 && TOTAL <= 227 * 1024, "shared memory of one CTA");
};

// Partial output of a piece: [ROWS][D] normalised, then [ROWS] log2 of the row's sum.  Slot 1 if it holds the unit's first tile.
template <int D, int ROWS>
__device__ __forceinline__ float* part8_at(float* part, int worker, int slot) {
  return part + (int64_t)(worker * 2 + slot) * (ROWS * (D + 1));
}

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 fp16 of a warp, transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
// 0x80 in every byte that is a NaN
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

template <int N>
__device__ __forceinline__ void lds(uint32_t* v, uint32_t addr) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
}

template <class T, int D, int NR, bool WIN>
__global__ void __launch_bounds__(NR == 1 ? 512 : 384, 1)
k_kv_attend8(const AttendArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using L = Attend8Shape<D, NR>;
  using S = typename L::template Tiles<WIN>;
  constexpr int NST = L::STAGES, KS = D / 16, WARPS = L::WARPS, THREADS = L::THREADS, ROWS = L::ROWS;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle goes by address bits
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = base + warp * (NST * L::STAGE), bars = base + L::BARS + warp * (8 * NST);
  float* s_o = reinterpret_cast<float*>(smem + L::O);
  float* s_m = reinterpret_cast<float*>(smem + L::STATS);
  float* s_l = s_m + ROWS * WARPS;
  float* s_r = s_l + ROWS * WARPS;
  int* s_walk = reinterpret_cast<int*>(smem + L::SMALL);
  int* s_sum = s_walk + 4;
  volatile int* abort = s_sum + 4 * WARPS;
  int* s_last = s_sum + 4 * WARPS + 1;

  if (base & 1023) {  // never: the swizzle would not hold
    if (tid == 0) a.status->code = TK_E_CUDA;
    return;
  }
  if (lane < NST) bar_init(bars + 8 * lane, 1);
  if (tid == 0) {
    *abort = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k));
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v));
  }
  fence_bar_init();
  Plan plan;
  const int total = make_plan<S, THREADS, 1, D>(a, plan, s_sum, s_walk);
  __syncthreads();

  const int me = blockIdx.x;
  // The walk and its pieces are in shared memory, where they cost no registers: the first thread goes on to
  // the next piece as one begins, the other warps ask for it when they have done their steps.
  Piece* s_piece = reinterpret_cast<Piece*>(smem + L::PIECES);
  Walk<S>* walk = reinterpret_cast<Walk<S>*>(s_piece + 2);
  static_assert(sizeof(Walk<S>) <= 192, "room for the walk");
  if (tid == 0) {
    walk->plan = plan;
    walk->from = me * plan.share;
    walk->to = min(total, walk->from + plan.share);
    walk->r = walk->from < total ? s_walk[0] : (int)a.R;
    walk->u = walk->from < total ? s_walk[1] : total;
    walk->loaded = false;
    walk->next(a, s_piece[0]);
  }
  __syncthreads();

  // ---- loads of the warp's steps: step i of a piece is its step number step0 + WARPS i
  uint32_t issued = 0, used = 0;  // stages of the ring, over all pieces
  bool ok = true;                 // no wait has given up: else the warp has no more steps
  int step0 = 0, n = 0, next = 0, window = 0;
  int id0 = 0, id1 = 0, id2 = 0;  // block ids of steps `window`, + 32 and + 64 + lane
  float2 sc0 = {0.f, 0.f}, sc1 = {0.f, 0.f};  // (ks, log2 of vs) of the first two
  const int32_t* row = nullptr;
  auto key_of = [&](const Piece& x, int i) {
    const int step = step0 + WARPS * i;
    return (WIN && step >= x.head ? step + x.skip : step) * A8_STEP;
  };
  auto id_of = [&](const Piece& x, int i) { return i + lane < n ? __ldg(row + (key_of(x, i + lane) >> a.log2_bs)) : -1; };
  // (of a block outside the cache zeros are read)
  auto scales_of = [&](const Piece& x, int id) {
    if (id < 0 || id >= a.n_blocks) return make_float2(0.f, E8_NONE);
    const int64_t at = (int64_t)id * a.hk + x.h;
    return make_float2(__ldg(a.k_scale + at), e8_log2(__ldg(a.v_scale + at)));
  };
  auto issue = [&](const Piece& x) {
    const int i = next - window;
    const int id = __shfl_sync(0xffffffffu, i < 32 ? id0 : id1, i & 31);
    const uint32_t st = issued % NST;
    if (elect_one()) {
      const int at = key_of(x, next) & ((1 << a.log2_bs) - 1);
      bar_expect(bars + 8 * st, L::STAGE);
      tma_load_4d(ring + st * L::STAGE, &map_k, bars + 8 * st, 0, at, x.h, id);
      tma_load_4d(ring + st * L::STAGE + L::TILE, &map_v, bars + 8 * st, 0, at, x.h, id);
    }
    __syncwarp();
    issued++;
    next++;
  };
  auto start = [&](const Piece& x) {
    const int steps = x.keys > 0 && ok ? min(x.hi * WARPS, (x.keys + A8_STEP - 1) / A8_STEP - (WIN ? x.skip : 0)) : 0;
    step0 = x.lo * WARPS + warp;
    n = max(0, (steps - step0 + WARPS - 1) / WARPS);
    next = window = 0;
    row = a.table + (int64_t)x.r * a.table_stride;
    id0 = id_of(x, 0);
    id1 = id_of(x, 32);
    id2 = id_of(x, 64);
    for (int i = 0; i < min(n, NST); i++) issue(x);
    sc0 = scales_of(x, id0);
    sc1 = scales_of(x, id1);
  };

  // ---- queries: of each 8 rows row g; of a thread's D / 4 neighbouring elements four are its share of a product
  uint32_t qb[NR][KS][2];
  float cq[NR][2];  // rows 2 t4 and + 1: scale log2(e) x what the elements are to be multiplied by
  auto fetch = [&](const Piece& x) {
#pragma unroll
    for (int r = 0; r < NR; r++) {
      const int rr = r * 8 + g, gr = x.row0 + rr, tok = by_group(a, gr);
      const T* src = static_cast<const T*>(a.q) + (x.t0 + tok) * a.q_stride + (x.h * a.group + gr - tok * a.group) * D + t4 * (D / 4);
      uint4 v[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; i++) v[i] = rr < x.rows ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
      float f = 1.f, back = 1.f;
      if (Pair<T>::BF) {
        // the largest finite element's exponent
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 8; i++) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(v)[i], lo = w & 0x7f80u, hi = (w >> 16) & 0x7f80u;
          if (lo < 0x7f80u) top = max(top, lo);
          if (hi < 0x7f80u) top = max(top, hi);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max((int)(top >> 7), 40), 254);  // below 2^-87 nothing is left
        f = __uint_as_float((uint32_t)(268 - e) << 23);     // 2^14 over the largest one's power of two
        back = __uint_as_float((uint32_t)(e - 14) << 23);
      }
      cq[r][0] = a.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t4);
      cq[r][1] = a.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t4 + 4);
#pragma unroll
      for (int i = 0; i < D / 8; i++) {
        uint32_t w = reinterpret_cast<const uint32_t*>(v)[i];
        if (Pair<T>::BF) {
          const float2 y = Pair<T>::up(*reinterpret_cast<const typename Pair<T>::type*>(&w));
          w = pack2<__half>(y.x * f, y.y * f);
        }
        qb[r][i >> 1][i & 1] = w;  // elements 2 i, 2 i + 1: product i / 2, first or second pair
      }
    }
  };

  int cur = 0;
  if (s_piece[0].valid) {
    start(s_piece[0]);
    fetch(s_piece[0]);
  }
  while (s_piece[cur].valid) {
    const Piece& p = s_piece[cur];
    const Piece& nx = s_piece[cur ^ 1];
    if (warp == 0) {
      if (lane == 0) walk->next(a, s_piece[cur ^ 1]);
      __syncwarp();
      asm volatile("bar.arrive 1, %0;" ::"n"(THREADS) : "memory");
    }
    // columns g * D / 8 + 2 j, + 1 of rows 2 t4, + 1
    float o[NR][KS][4], m[NR][2], l[NR][2], bound[NR][2];  // m is M, bound R
#pragma unroll
    for (int r = 0; r < NR; r++) {
      m[r][0] = m[r][1] = bound[r][0] = bound[r][1] = -E8_MOST;
      l[r][0] = l[r][1] = 0.f;
#pragma unroll
      for (int j = 0; j < KS; j++) o[r][j][0] = o[r][j][1] = o[r][j][2] = o[r][j][3] = 0.f;
    }

#pragma unroll 1
    for (int i = 0; i < n && ok; i++) {
      if (i == window + 32) {
        window += 32;
        id0 = id1;
        sc0 = sc1;
        id1 = id2;
        sc1 = scales_of(p, id1);
        id2 = id_of(p, i + 64);
      }
      const float ks = __shfl_sync(0xffffffffu, sc0.x, i & 31), lv = __shfl_sync(0xffffffffu, sc0.y, i & 31);
      const int k0 = key_of(p, i);
      const bool hidden = !(k0 + A8_STEP <= p.open && (!WIN || k0 >= p.shut || k0 + A8_STEP <= a.sinks));
      const uint32_t st = used % NST, s_k = ring + st * L::STAGE, s_v = s_k + L::TILE;
      ok = __all_sync(0xffffffffu, bar_wait(bars + 8 * st, (used / NST) & 1, abort)) != 0;
      if (!ok) break;
      used++;

      // keys g and g + 8; values: keys 2 t4, + 1, + 8, + 9, neighbouring columns from g * D / 8 on
      uint32_t kw[2][KS], vw[4][KS / 2];
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int key = j * 8 + g;
        if constexpr (D == 128) {
          lds<4>(kw[j], s_k + key * 128 + (((2 * t4) ^ (key & 7)) << 4));
          lds<4>(kw[j] + 4, s_k + key * 128 + (((2 * t4 + 1) ^ (key & 7)) << 4));
        } else {
          lds<4>(kw[j], s_k + key * 64 + ((t4 ^ ((key >> 1) & 3)) << 4));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int key = 2 * t4 + (e & 1) + (e >> 1) * 8;
        if constexpr (D == 128) lds<4>(vw[e], s_v + key * 128 + ((g ^ (key & 7)) << 4));
        else lds<2>(vw[e], s_v + key * 64 + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
      }
      // scores of keys g (0, 1) and g + 8 (2, 3), rows 2 t4, + 1
      float s[NR][4];
#pragma unroll
      for (int r = 0; r < NR; r++) s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        const uint32_t ka[4] = {e4m3_lo(kw[0][k]), e4m3_lo(kw[1][k]), e4m3_hi(kw[0][k]), e4m3_hi(kw[1][k])};
#pragma unroll
        for (int r = 0; r < NR; r++) mma16816(s[r], ka, qb[r][k][0], qb[r][k][1]);
      }
      __syncwarp();  // the stage has been read
      if (next < n) issue(p);

      uint32_t bits[NR][2];  // keys g and g + 8: bits 0 and 8
      if (hidden) {
#pragma unroll
        for (int r = 0; r < NR; r++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int rr = r * 8 + 2 * t4 + e;
            Seen<WIN> seen;
            seen.set(a, p, rr < p.rows, rr < p.rows ? by_group(a, p.row0 + rr) : 0);
            bits[r][e] = seen.bits(k0) >> g;
            if (!(bits[r][e] & 1)) s[r][e] = -INFINITY;
            if (!(bits[r][e] & 256)) s[r][2 + e] = -INFINITY;
          }
      }
      uint32_t pb[NR][2];
#pragma unroll
      for (int r = 0; r < NR; r++) {
        // with the least normal number a hidden key's -infinity stays that
        const float c0 = fmaxf(cq[r][0] * ks, 1.17549435e-38f), c1 = fmaxf(cq[r][1] * ks, 1.17549435e-38f);
        float x0 = fmaxf(s[r][0], s[r][2]) * c0, x1 = fmaxf(s[r][1], s[r][3]) * c1;
        if (__any_sync(0xffffffffu, x0 > m[r][0] || x1 > m[r][1] || x0 + lv > bound[r][0] || x1 + lv > bound[r][1])) {
#pragma unroll
          for (int e = 4; e < 32; e *= 2) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, e));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, e));
          }
          // the factor that a new bound brings with it
          auto pass = [](float x, float& at) {
            if (!(x > at)) return 1.f;
            const float was = at;
            at = x + 8.f;
            return exp2_fast(was - at);
          };
          l[r][0] *= pass(x0, m[r][0]);
          l[r][1] *= pass(x1, m[r][1]);
          const float f0 = pass(x0 + lv, bound[r][0]), f1 = pass(x1 + lv, bound[r][1]);
#pragma unroll
          for (int j = 0; j < KS; j++) {
            o[r][j][0] *= f0;
            o[r][j][1] *= f1;
            o[r][j][2] *= f0;
            o[r][j][3] *= f1;
          }
        }
        const float d0 = e8_shift(lv, m[r][0], bound[r][0]), d1 = e8_shift(lv, m[r][1], bound[r][1]);
        const float to0 = d0 - m[r][0], to1 = d1 - m[r][1];
        const float p0 = exp2_fast(fmaf(s[r][0], c0, to0)), p1 = exp2_fast(fmaf(s[r][1], c1, to1)),
                    p2 = exp2_fast(fmaf(s[r][2], c0, to0)), p3 = exp2_fast(fmaf(s[r][3], c1, to1));
        l[r][0] = fmaf(p0 + p2, exp2_fast(-d0), l[r][0]);
        l[r][1] = fmaf(p1 + p3, exp2_fast(-d1), l[r][1]);
        pb[r][0] = transpose8x8(pack2<__half>(p0, p1));
        pb[r][1] = transpose8x8(pack2<__half>(p2, p3));
      }

      // values of keys that a row does not see have no influence on it: NaN become 0, and come
      // back for the rows that see them.  (0x80 marks a NaN byte.)
      if (hidden) {
        uint32_t bad = 0;
#pragma unroll
        for (int e = 0; e < 4; e++)
#pragma unroll
          for (int j = 0; j < KS / 2; j++) bad |= e4m3_nan(vw[e][j]);
        if (__any_sync(0xffffffffu, bad != 0)) {
          // columns x keys that are NaN, as a matrix of ones, times keys x rows that see them
#pragma unroll
          for (int r = 0; r < NR; r++) {
            const uint32_t b0 = transpose8x8((bits[r][0] & 1 ? 0x3c00u : 0u) | (bits[r][1] & 1 ? 0x3c000000u : 0u)),
                           b1 = transpose8x8((bits[r][0] & 256 ? 0x3c00u : 0u) | (bits[r][1] & 256 ? 0x3c000000u : 0u));
#pragma unroll
            for (int j = 0; j < KS; j++) {
              uint32_t one[4];
#pragma unroll
              for (int x = 0; x < 4; x++) {
                const int e = (x >> 1) * 2, at = 8 * ((2 * j + (x & 1)) & 3) + 7;
                one[x] = ((e4m3_nan(vw[e][j >> 1]) >> at) & 1 ? 0x3c00u : 0u) | ((e4m3_nan(vw[e + 1][j >> 1]) >> at) & 1 ? 0x3c000000u : 0u);
              }
              float met[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(met, one, b0, b1);
#pragma unroll
              for (int x = 0; x < 4; x++)
                if (met[x] > 0.f) o[r][j][x] = __int_as_float(0x7fffffff);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; e++)
#pragma unroll
            for (int j = 0; j < KS / 2; j++) vw[e][j] &= ~((e4m3_nan(vw[e][j]) >> 7) * 255u);
        }
      }
#pragma unroll
      for (int j = 0; j < KS; j++) {  // two columns: bytes 2 (j & 1), + 1 of word j / 2
        const uint32_t pick = j & 1 ? 0x7362u : 0x5140u;
        const uint32_t x = __byte_perm(vw[0][j >> 1], vw[1][j >> 1], pick), y = __byte_perm(vw[2][j >> 1], vw[3][j >> 1], pick);
        const uint32_t va[4] = {e4m3_lo(x), e4m3_hi(x), e4m3_lo(y), e4m3_hi(y)};
#pragma unroll
        for (int r = 0; r < NR; r++) mma16816(o[r][j], va, pb[r][0], pb[r][1]);
      }
    }

    // ---- the warps' outputs become the piece's
#pragma unroll
    for (int r = 0; r < NR; r++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float x = l[r][e];
#pragma unroll
        for (int d = 4; d < 32; d *= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (g == 0) {
          s_m[(r * 8 + 2 * t4 + e) * WARPS + warp] = m[r][e];
          s_l[(r * 8 + 2 * t4 + e) * WARPS + warp] = x;
          s_r[(r * 8 + 2 * t4 + e) * WARPS + warp] = bound[r][e];
        }
      }
    if (warp != 0) asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
    // What is asked after a whole piece's last barrier is in registers: the first warp may have begun the next piece by
    // then, and be writing the one after that over this one.
    const bool whole = p.pieces == 1;
    const int groups = NR == 1 ? 1 : (p.rows + 7) / 8;
    float* part = part8_at<D, ROWS>(a.part, me, p.lo == 0);
#pragma unroll
    for (int r = 0; r < NR; r++) {
      if (r >= groups) break;
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float* dst = s_o + (warp * 8 + 2 * t4 + e) * L::O_ROW + g * L::O_GROUP;
#pragma unroll
        for (int j = 0; j < KS; j += 2)
          *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[r][j][e], o[r][j][2 + e], o[r][j + 1][e], o[r][j + 1][2 + e]);
      }
      if (r == 0 && nx.valid) start(nx);
      __syncthreads();
      for (int x = tid; x < min(p.rows - r * 8, 8) * (D / 4); x += THREADS) {
        const int in = x / (D / 4), rr = r * 8 + in, col = (x % (D / 4)) * 4;
        float M = -E8_MOST, R = -E8_MOST, sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; w++) {
          M = fmaxf(M, s_m[rr * WARPS + w]);
          R = fmaxf(R, s_r[rr * WARPS + w]);
        }
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; w++) {
          const float lw = s_l[rr * WARPS + w];
          if (lw == 0.f) continue;  // the warp saw nothing
          sum = fmaf(exp2_fast(s_m[rr * WARPS + w] - M), lw, sum);
          const float f = exp2_fast(s_r[rr * WARPS + w] - R);
          const float4 z = *reinterpret_cast<const float4*>(s_o + (w * 8 + in) * L::O_ROW + col / (D / 8) * L::O_GROUP + col % (D / 8));
          y.x = fmaf(f, z.x, y.x);
          y.y = fmaf(f, z.y, y.y);
          y.z = fmaf(f, z.z, y.z);
          y.w = fmaf(f, z.w, y.w);
        }
        const bool none = sum == 0.f;
        // (in two factors: of scales from 2^127 on it may be more than fp32 has)
        const float half = exp2f(0.5f * (R - E8_TOP - M)), inv = none ? 0.f : half / sum;
        y = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                 : make_float4(y.x * inv * half, y.y * inv * half, y.z * inv * half, y.w * inv * half);
        const float log2sum = none ? -INFINITY : M + log2f(sum);
        if (whole) {
          const int gr = p.row0 + rr, tok = by_group(a, gr);
          const int64_t at = (int64_t)(p.t0 + tok) * a.hq + p.h * a.group + (gr - tok * a.group);
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + col) = make_uint2(pack2<T>(y.x, y.y), pack2<T>(y.z, y.w));
          if (a.lse && col == 0) a.lse[at] = log2sum * 0.69314718055994531f;
        } else {
          __stcg(reinterpret_cast<float4*>(part + rr * D + col), y);
          if (col == 0) __stcg(part + ROWS * D + rr, log2sum);
        }
      }
      __syncthreads();  // the outputs have been read
    }
    if (nx.valid) fetch(nx);
    if (!whole) {
      // The last of a unit's pieces to be ready joins them, always in the same order.
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned before = atomicAdd(a.counters + 2 * p.first, 1u);
        *s_last = before == (unsigned)p.pieces - 1;
        if (*s_last) a.counters[2 * p.first] = 0;  // all have come by
        __threadfence();
      }
      __syncthreads();
      if (*s_last && !*abort) {
        for (int x = tid; x < p.rows * (D / 4); x += THREADS) {
          const int rr = x / (D / 4), col = (x % (D / 4)) * 4;
          float top = -INFINITY, sum = 0.f;
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int j0 = 0; j0 < p.pieces; j0 += 8) {
            float e[8];
            float4 z[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
              const int pc = j0 + j;
              const float* src = part8_at<D, ROWS>(a.part, p.first + pc, pc == 0);
              e[j] = pc < p.pieces ? __ldcg(src + ROWS * D + rr) : -INFINITY;
              z[j] = pc < p.pieces ? __ldcg(reinterpret_cast<const float4*>(src + rr * D + col)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float high = top;
#pragma unroll
            for (int j = 0; j < 8; j++) high = fmaxf(high, e[j]);
            const float f = top == -INFINITY ? 0.f : exp2_fast(top - high);
            sum *= f;
            y.x *= f; y.y *= f; y.z *= f; y.w *= f;
            top = high;
#pragma unroll
            for (int j = 0; j < 8; j++) {
              if (e[j] == -INFINITY) continue;  // a piece without weight
              const float w = exp2_fast(e[j] - top);
              sum += w;
              y.x = fmaf(w, z[j].x, y.x);
              y.y = fmaf(w, z[j].y, y.y);
              y.z = fmaf(w, z[j].z, y.z);
              y.w = fmaf(w, z[j].w, y.w);
            }
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const int gr = p.row0 + rr, tok = by_group(a, gr);
          const int64_t at = (int64_t)(p.t0 + tok) * a.hq + p.h * a.group + (gr - tok * a.group);
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + col) =
              make_uint2(pack2<T>(y.x * inv, y.y * inv), pack2<T>(y.z * inv, y.w * inv));
          if (a.lse && col == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        }
      }
      __syncthreads();  // s_last and the piece have been read
    }
    cur ^= 1;
  }
  // given up: the copies in flight land before the CTA ends
  if (!ok)
    for (; used != issued; used++)
      for (uint32_t i = 0; i < 1u << 16 && !bar_try(bars + 8 * (used % NST), (used / NST) & 1); i++) {}
  if (*abort && lane == 0) {
    atomicExch(&a.status->code, TK_E_TIMEOUT);
    a.status->request = -1;
  }
}

template <class T, int D, int NR, bool WIN>
static cudaError_t attend8_launch(const AttendArgs& a, const tk_kv_cache* cache, int grid, cudaStream_t st) {
  constexpr int bytes = Attend8Shape<D, NR>::TOTAL;
  static bool set[64];  // by device
  if (cache->device >= 64 || !set[cache->device]) {
    const cudaError_t e = cudaFuncSetAttribute(k_kv_attend8<T, D, NR, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (cache->device < 64) set[cache->device] = true;
  }
  k_kv_attend8<T, D, NR, WIN><<<grid, Attend8Shape<D, NR>::THREADS, bytes, st>>>(a, cache->map_k16, cache->map_v16);
  return cudaGetLastError();
}

template <class T, int D, bool WIN>
static cudaError_t attend8_rows(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  return rows <= 8 ? attend8_launch<T, D, 1, WIN>(a, cache, grid, st) : attend8_launch<T, D, 2, WIN>(a, cache, grid, st);
}

template <class T, int D>
static cudaError_t attend8_pick(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  return a.window < INT32_MAX ? attend8_rows<T, D, true>(a, cache, rows, grid, st) : attend8_rows<T, D, false>(a, cache, rows, grid, st);
}

cudaError_t attend8(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  if (rows > 16) return attend8_many(a, cache, rows, grid, st);
  if (cache->type == TK_BF16)
    return cache->head_dim == 64 ? attend8_pick<__nv_bfloat16, 64>(a, cache, rows, grid, st)
                                 : attend8_pick<__nv_bfloat16, 128>(a, cache, rows, grid, st);
  return cache->head_dim == 64 ? attend8_pick<__half, 64>(a, cache, rows, grid, st) : attend8_pick<__half, 128>(a, cache, rows, grid, st);
}

}  // namespace tk
