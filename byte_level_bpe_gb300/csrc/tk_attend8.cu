// tk_attend8.cu -- attention over a paged cache in 8 bits (tk_kv_attend, tk_kv_attend_window):
// o = sum_j softmax_j(scale ks_j q.k_j) vs_j v_j, k_j and v_j e4m3, ks_j and vs_j their block's scales.
//
// e4m3 is a subset of fp16, so keys and values enter the products exactly, as fp16, whatever the
// queries' type.  Queries of bf16 become fp16 with a power of two for each row that brings their largest element to
// 2^14: exact but for elements 2^-28 below it, which lose less than fp32's sums do.  The scales
// stay outside: the keys' is a factor of the scores (a step of 16 keys lies in one block), the
// values' of the weights, relative to the largest so far:
//   x_j = c ks_j (q.k_j), c = scale log2(e);  p_j = 2^(x_j - m + 7), l += p_j;
//   w_j = p_j vs_j 2^-E rounded to fp16, O += w_j v_j; o = 2^E O / l.
// m is a running maximum that the weights may pass by 2^8, E the exponent of the largest vs so far: w < 2^15.
// A weight that fp16 loses is 2^-31 of the largest and less.
//
// Up to 16 rows (query heads of a key head x tokens) memory is the bound by far, and the tensor cores' 16-bit
// operands would cost more shared memory traffic than the keys and values themselves (the two products of 64 keys of
// head_dim 128 read 64 KB, which takes the 8-bit tile 700 cycles to arrive and them 512, and the conversion
// 64 KB more).  So a warp's products are those of its registers (m16n8k16): it reads a key's 16 bytes as
// they are, four neighbouring elements being one thread's share of a product of 16, which may be any 16 as long as
// the queries take the same; of the values a thread has four keys' 16 bytes, whose bytes it pairs up.
// Nothing is written to shared memory but what TMA brings.
#include "tk_attend.cuh"

namespace tk {

constexpr int A8_WARPS = 8, A8_THREADS = A8_WARPS * 32;
constexpr int A8_SUB = 16;  // keys of a product: they lie in one block
constexpr int A8_UNIT_COST = 1, A8_MIN_SHARE = 2, A8_SNAP = 1;
constexpr float A8_UP = 7.f;

// A warp has a ring of its own: STAGES steps of keys and values.
// A step, one warp's, is SUBS times 16 keys.
template <int D, int MT>
struct Attend8Shape {
  static constexpr int ROWS = 16 * MT;
  static constexpr int SUBS = MT == 1 ? 2 : 1, STEP = SUBS * A8_SUB;
  static constexpr int TILE = STEP * D, STAGE = 2 * TILE, STAGES = 16 * 1024 / STAGE;  // 16 KB a warp
  static constexpr int DIMS = D / 4;                      // neighbouring columns that a thread has of an output
  static constexpr int O_GROUP = DIMS + 4, O_ROW = 4 * O_GROUP;  // floats; quarter-warps meet no bank twice
  static constexpr int O = A8_WARPS * STAGES * STAGE;     // [warp][16][O_ROW] outputs of the warps, for one 16 rows at a time
  static constexpr int Q = O + A8_WARPS * 16 * O_ROW * 4; // MT = 2: the queries as the products want them
  static constexpr int STATS = Q + (MT > 1 ? MT * (D / 16) * 512 : 0);  // [MT][warp][16] m, l; [warp] E
  static constexpr int BARS = STATS + (2 * MT * 16 + 2) * A8_WARPS * 4;
  static constexpr int SMALL = BARS + 8 * A8_WARPS * STAGES;
  static constexpr int PIECES = SMALL + 16 + 4 * A8_WARPS * 4 + 16;  // this one and the next one; the walk
  static constexpr int TOTAL = PIECES + 2 * (int)sizeof(Piece) + 192;
  template <bool WIN>
  using Tiles = Tiling<ROWS, STEP, A8_WARPS, WIN, A8_UNIT_COST, A8_MIN_SHARE, A8_SNAP, 2, true>;
  static_assert(SMALL % 8 == 0 && TOTAL <= 227 * 1024, "shared memory of one CTA");
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
// 0x80 in every byte that is a NaN
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

template <int N>
__device__ __forceinline__ void lds(uint32_t* v, uint32_t addr) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
}

template <class T, int D, int MT, bool WIN>
__global__ void __launch_bounds__(A8_THREADS, 1)
k_kv_attend8(const AttendArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using L = Attend8Shape<D, MT>;
  using S = typename L::template Tiles<WIN>;
  constexpr int NST = L::STAGES, KS = D / 16, NT = D / 8, ROWS = L::ROWS, DIMS = L::DIMS, SUBS = L::SUBS, STEP = L::STEP;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle goes by address bits
  const uint32_t base = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = base + warp * (NST * L::STAGE), bars = base + L::BARS + warp * (8 * NST);
  float* s_o = reinterpret_cast<float*>(smem + L::O);
  float* s_m = reinterpret_cast<float*>(smem + L::STATS);  // [MT][16][warp]
  float* s_l = s_m + MT * 16 * A8_WARPS;
  int* s_e = reinterpret_cast<int*>(s_l + MT * 16 * A8_WARPS);
  int* s_walk = reinterpret_cast<int*>(smem + L::SMALL);
  int* s_sum = s_walk + 4;
  volatile int* abort = s_sum + 4 * A8_WARPS;
  int* s_last = s_sum + 4 * A8_WARPS + 1;

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
  const int total = make_plan<S, A8_THREADS, 1, D>(a, plan, s_sum, s_walk);
  __syncthreads();

  const int me = blockIdx.x;
  // The walk and its pieces are in shared memory, where they cost no registers: the first thread goes on to
  // the next piece as one begins, the other warps ask for it when they have done their steps.
  Piece* s_piece = reinterpret_cast<Piece*>(smem + L::PIECES);
  Walk<S>* walk = reinterpret_cast<Walk<S>*>(s_piece + 2);
  static_assert(sizeof(Walk<S>) <= 192 && L::PIECES % 8 == 0, "room for the walk");
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

  // ---- loads of the warp's steps: step i of a piece is its step number step0 + 8 i
  uint32_t issued = 0, used = 0;  // stages of the ring, over all pieces
  bool ok = true;                 // no wait has given up: else the warp has no more steps
  int step0 = 0, n = 0, next = 0, window = 0;
  // lane: 16 keys each from step `window` on, their block ids and those of the next 32 and 32 times 16
  constexpr int AHEAD = 32 / SUBS;  // steps of 32 lanes
  int id0 = 0, id1 = 0, id2 = 0;
  float2 sc0 = {0.f, 0.f}, sc1 = {0.f, 0.f};  // (ks, vs) of the first two
  const int32_t* row = nullptr;
  auto key_of = [&](const Piece& x, int i) {
    const int step = step0 + A8_WARPS * i;
    return (WIN && step >= x.head ? step + x.skip : step) * STEP;
  };
  // (of a block outside the cache zeros are read, and of keys past the end)
  auto id_of = [&](const Piece& x, int i) {
    const int at = i + lane / SUBS, key = key_of(x, at) + lane % SUBS * A8_SUB;
    return at < n && key < x.keys ? __ldg(row + (key >> a.log2_bs)) : -1;
  };
  auto scales_of = [&](const Piece& x, int id) {
    if (id < 0 || id >= a.n_blocks) return make_float2(0.f, 0.f);
    const int64_t at = (int64_t)id * a.hk + x.h;
    return make_float2(__ldg(a.k_scale + at), __ldg(a.v_scale + at));
  };
  auto issue = [&](const Piece& x) {
    const int i = next - window, sub = lane % SUBS;
    const int id = __shfl_sync(0xffffffffu, i < AHEAD ? id0 : id1, (i * SUBS + sub) & 31);
    const uint32_t st = issued % NST;
    if (lane == 0) bar_expect(bars + 8 * st, L::STAGE);
    __syncwarp();
    if (lane < 2 * SUBS) {  // keys, then values
      const int at = (key_of(x, next) + sub * A8_SUB) & ((1 << a.log2_bs) - 1);
      tma_load_4d(ring + st * L::STAGE + lane * (A8_SUB * D), lane < SUBS ? &map_k : &map_v, bars + 8 * st, 0, at, x.h, id);
    }
    __syncwarp();
    issued++;
    next++;
  };
  auto start = [&](const Piece& x) {
    const int steps = x.keys > 0 && ok ? min(x.hi * A8_WARPS, (x.keys + STEP - 1) / STEP - (WIN ? x.skip : 0)) : 0;
    step0 = x.lo * A8_WARPS + warp;
    n = max(0, (steps - step0 + A8_WARPS - 1) / A8_WARPS);
    next = window = 0;
    row = a.table + (int64_t)x.r * a.table_stride;
    id0 = id_of(x, 0);
    id1 = id_of(x, AHEAD);
    id2 = id_of(x, 2 * AHEAD);
    for (int i = 0; i < min(n, NST); i++) issue(x);
    sc0 = scales_of(x, id0);
    sc1 = scales_of(x, id1);
  };

  // ---- queries: rows g and g + 8 of each 16; of its DIMS neighbouring elements four are a thread's share of a product
  uint32_t qa[MT == 1 ? KS : 1][4];
  float qs[MT][2];  // what the elements were divided by
  auto fetch = [&](const Piece& x) {
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const int rr = mt * 16 + half * 8 + g, gr = x.row0 + rr, tok = gr / a.group;
        const T* src = static_cast<const T*>(a.q) + (x.t0 + tok) * a.q_stride + (x.h * a.group + gr - tok * a.group) * D + t4 * DIMS;
        uint4 v[DIMS / 8];
#pragma unroll
        for (int i = 0; i < DIMS / 8; i++) v[i] = rr < x.rows ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
        float f = 1.f, back = 1.f;
        if (Pair<T>::BF) {
          // the largest finite element's exponent
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < DIMS / 2; i++) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(v)[i], lo = w & 0x7f80u, hi = (w >> 16) & 0x7f80u;
            if (lo < 0x7f80u) top = max(top, lo);
            if (hi < 0x7f80u) top = max(top, hi);
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = min(max((int)(top >> 7), 40), 254);  // below 2^-87 nothing is left
          f = __uint_as_float((uint32_t)(268 - e) << 23);     // 2^(14 - (e - 127)), which 253 is the most of
          back = __uint_as_float((uint32_t)(e - 14) << 23);
        }
        qs[mt][half] = back;
#pragma unroll
        for (int i = 0; i < DIMS / 2; i++) {
          uint32_t w = reinterpret_cast<const uint32_t*>(v)[i];
          if (Pair<T>::BF) {
            const float2 y = Pair<T>::up(*reinterpret_cast<const typename Pair<T>::type*>(&w));
            w = pack2<__half>(y.x * f, y.y * f);
          }
          // word i = elements 2 i, 2 i + 1: product i / 2, first or second pair
          const int reg = (i & 1) * 2 + half;
          if constexpr (MT == 1) qa[i >> 1][reg] = w;
          else if (warp == 0) reinterpret_cast<uint32_t*>(smem + L::Q)[((mt * KS + (i >> 1)) * 32 + lane) * 4 + reg] = w;
        }
      }
    }
  };

  int cur = 0;
  if (s_piece[0].valid) {
    start(s_piece[0]);
    fetch(s_piece[0]);
  }
  if (MT > 1) __syncthreads();
  while (s_piece[cur].valid) {
    const Piece& p = s_piece[cur];
    const Piece& nx = s_piece[cur ^ 1];
    if (warp == 0) {
      if (lane == 0) walk->next(a, s_piece[cur ^ 1]);
      __syncwarp();
      asm volatile("bar.arrive 1, %0;" ::"n"(A8_THREADS) : "memory");
    }
    float o[MT][NT][4];
    float m[MT][2], l[MT][2];
    int E = -1000;
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < NT; j++) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
    }
    float cr[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      cr[mt][0] = a.scale_log2 * qs[mt][0];
      cr[mt][1] = a.scale_log2 * qs[mt][1];
    }

#pragma unroll 1
    for (int i = 0; i < n && ok; i++) {
      if (i == window + AHEAD) {
        window += AHEAD;
        id0 = id1;
        sc0 = sc1;
        id1 = id2;
        sc1 = scales_of(p, id1);
        id2 = id_of(p, i + 2 * AHEAD);
      }
      float ks[SUBS], vs[SUBS];
#pragma unroll
      for (int u = 0; u < SUBS; u++) {
        ks[u] = __shfl_sync(0xffffffffu, sc0.x, (i * SUBS + u) & 31);
        vs[u] = __shfl_sync(0xffffffffu, sc0.y, (i * SUBS + u) & 31);
      }
      const int k0 = key_of(p, i);
      const bool hidden = !(k0 + STEP <= p.open && (!WIN || k0 >= p.shut || k0 + STEP <= a.sinks));
      const uint32_t st = used % NST, s_k = ring + st * L::STAGE, s_v = s_k + L::TILE;
      ok = __all_sync(0xffffffffu, bar_wait(bars + 8 * st, (used / NST) & 1, abort)) != 0;
      if (!ok) break;
      used++;

      // scores
      float s[MT][2 * SUBS][4];
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int e = 0; e < 8 * SUBS; e++) s[mt][e >> 2][e & 3] = 0.f;
      uint32_t kw[2 * SUBS][D / 16];
#pragma unroll
      for (int j = 0; j < 2 * SUBS; j++) {
        const int key = j * 8 + g;
        if constexpr (D == 128) {
          lds<4>(kw[j], s_k + key * 128 + (((2 * t4) ^ (key & 7)) << 4));
          lds<4>(kw[j] + 4, s_k + key * 128 + (((2 * t4 + 1) ^ (key & 7)) << 4));
        } else {
          lds<4>(kw[j], s_k + key * 64 + ((t4 ^ ((key >> 1) & 3)) << 4));
        }
      }
#pragma unroll
      for (int k = 0; k < KS; k++) {
        uint32_t q4[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
          if constexpr (MT == 1) {
#pragma unroll
            for (int e = 0; e < 4; e++) q4[mt][e] = qa[k][e];
          } else {
            lds<4>(q4[mt], base + L::Q + ((mt * KS + k) * 32 + lane) * 16);
          }
        }
#pragma unroll
        for (int j = 0; j < 2 * SUBS; j++) {
          const uint32_t b0 = e4m3_lo(kw[j][k]), b1 = e4m3_hi(kw[j][k]);
#pragma unroll
          for (int mt = 0; mt < MT; mt++) mma16816(s[mt][j], q4[mt], b0, b1);
        }
      }
      // values: of each 16 keys 2 t4, + 1, + 8, + 9; neighbouring columns g * NT ..
      uint32_t vw[SUBS][4][NT / 4];
#pragma unroll
      for (int u = 0; u < SUBS; u++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int key = u * 16 + 2 * t4 + (e & 1) + (e >> 1) * 8;
          if constexpr (D == 128) lds<4>(vw[u][e], s_v + key * 128 + ((g ^ (key & 7)) << 4));
          else lds<2>(vw[u][e], s_v + key * 64 + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
        }
      __syncwarp();  // the stage has been read
      if (next < n) issue(p);

      float largest = vs[0];
      if (SUBS > 1) largest = fmaxf(vs[0], vs[SUBS - 1]);
      const int ev = largest > 0.f ? (int)((__float_as_uint(largest) >> 23) & 255) - 126 : -1000;  // vs <= 2^ev
      const bool larger = ev > E;
      float shrink = 1.f;
      if (larger) {
        shrink = E < -500 ? 0.f : exp2f((float)(E - ev));
        E = ev;
      }
      // 2^-E in two factors: it may be below the least normal number
      const float down = E < -500 ? 0.f : __uint_as_float((uint32_t)(127 - E / 2) << 23),
                  down2 = E < -500 ? 0.f : __uint_as_float((uint32_t)(127 - (E - E / 2)) << 23);
      float vn[SUBS];
#pragma unroll
      for (int u = 0; u < SUBS; u++) vn[u] = vs[u] * down * down2;
      uint32_t w4[MT][SUBS][4], bits[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
#pragma unroll
        for (int j = 0; j < 2 * SUBS; j++) {
          const float c0 = cr[mt][0] * ks[j >> 1], c1 = cr[mt][1] * ks[j >> 1];
          s[mt][j][0] *= c0;
          s[mt][j][1] *= c0;
          s[mt][j][2] *= c1;
          s[mt][j][3] *= c1;
        }
        if (hidden) {
#pragma unroll
          for (int half = 0; half < 2; half++) {
            const int rr = mt * 16 + half * 8 + g;
            Seen<WIN> seen;
            seen.set(a, p, rr < p.rows, rr < p.rows ? (p.row0 + rr) / a.group : 0);
            bits[mt][half] = seen.bits(k0);
#pragma unroll
            for (int j = 0; j < 2 * SUBS; j++)
#pragma unroll
              for (int e = 0; e < 2; e++)
                if (!((bits[mt][half] >> (j * 8 + 2 * t4 + e)) & 1)) s[mt][j][half * 2 + e] = -INFINITY;
          }
        }
        float mx[2];
        bool grow = false;
#pragma unroll
        for (int half = 0; half < 2; half++) {
          float x = fmaxf(s[mt][0][2 * half], s[mt][0][2 * half + 1]);
#pragma unroll
          for (int j = 1; j < 2 * SUBS; j++) x = max3(x, s[mt][j][2 * half], s[mt][j][2 * half + 1]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          mx[half] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          grow |= mx[half] > m[mt][half] && !(mx[half] - m[mt][half] <= 8.f);
        }
        if (__any_sync(0xffffffffu, grow || larger)) {
          float f[2];
#pragma unroll
          for (int half = 0; half < 2; half++) {
            const bool up = mx[half] > m[mt][half] && !(mx[half] - m[mt][half] <= 8.f);
            const float by = up ? exp2_fast(m[mt][half] - mx[half]) : 1.f;
            if (up) m[mt][half] = mx[half];
            l[mt][half] *= by;
            f[half] = by * shrink;
          }
#pragma unroll
          for (int j = 0; j < NT; j++) {
            o[mt][j][0] *= f[0];
            o[mt][j][1] *= f[0];
            o[mt][j][2] *= f[1];
            o[mt][j][3] *= f[1];
          }
        }
        const float m0 = m[mt][0] == -INFINITY ? 0.f : m[mt][0] - A8_UP, m1 = m[mt][1] == -INFINITY ? 0.f : m[mt][1] - A8_UP;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * SUBS; j++) {
          const float p0 = exp2_fast(s[mt][j][0] - m0), p1 = exp2_fast(s[mt][j][1] - m0), p2 = exp2_fast(s[mt][j][2] - m1),
                      p3 = exp2_fast(s[mt][j][3] - m1);
          l0 += p0 + p1;
          l1 += p2 + p3;
          w4[mt][j >> 1][2 * (j & 1)] = pack2<__half>(p0 * vn[j >> 1], p1 * vn[j >> 1]);
          w4[mt][j >> 1][2 * (j & 1) + 1] = pack2<__half>(p2 * vn[j >> 1], p3 * vn[j >> 1]);
        }
        l[mt][0] += l0;
        l[mt][1] += l1;
      }

      // values of keys that a row does not see have no influence on it: NaN become 0, and come
      // back for the rows that see them.  (0x80 marks a NaN byte.)
      uint32_t bad = 0;
      if (hidden) {
#pragma unroll
        for (int u = 0; u < SUBS; u++)
#pragma unroll
          for (int e = 0; e < 4; e++)
#pragma unroll
            for (int j = 0; j < NT / 4; j++) bad |= e4m3_nan(vw[u][e][j]);
        bad = __any_sync(0xffffffffu, bad != 0);
      }
      if (bad) {
#pragma unroll
        for (int u = 0; u < SUBS; u++) {
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            // rows x keys that are seen, as a matrix of ones, times keys x columns that are NaN
            uint32_t one[4];
#pragma unroll
            for (int x = 0; x < 4; x++) {
              const uint32_t b = bits[mt][x & 1] >> (u * 16 + (x >> 1) * 8 + 2 * t4);
              one[x] = (b & 1 ? 0x3c00u : 0u) | (b & 2 ? 0x3c000000u : 0u);
            }
#pragma unroll
            for (int j = 0; j < NT; j++) {
              auto ones = [&](uint32_t x, uint32_t y) {
                return ((e4m3_nan(x) >> (8 * (j & 3) + 7)) & 1 ? 0x3c00u : 0u) | ((e4m3_nan(y) >> (8 * (j & 3) + 7)) & 1 ? 0x3c000000u : 0u);
              };
              float met[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(met, one, ones(vw[u][0][j >> 2], vw[u][1][j >> 2]), ones(vw[u][2][j >> 2], vw[u][3][j >> 2]));
#pragma unroll
              for (int x = 0; x < 4; x++)
                if (met[x] > 0.f) o[mt][j][x] = __int_as_float(0x7fffffff);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; e++)
#pragma unroll
            for (int j = 0; j < NT / 4; j++) vw[u][e][j] &= ~((e4m3_nan(vw[u][e][j]) >> 7) * 255u);
        }
      }
#pragma unroll
      for (int u = 0; u < SUBS; u++) {
#pragma unroll
        for (int j = 0; j < NT / 2; j++) {  // two columns: bytes 2 (j & 1), + 1 of word j / 2
          const uint32_t pick = j & 1 ? 0x7362u : 0x5140u;
          const uint32_t x = __byte_perm(vw[u][0][j >> 1], vw[u][1][j >> 1], pick), y = __byte_perm(vw[u][2][j >> 1], vw[u][3][j >> 1], pick);
          const uint32_t b00 = e4m3_lo(x), b01 = e4m3_lo(y), b10 = e4m3_hi(x), b11 = e4m3_hi(y);
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            mma16816(o[mt][2 * j], w4[mt][u], b00, b01);
            mma16816(o[mt][2 * j + 1], w4[mt][u], b10, b11);
          }
        }
      }
    }

    // ---- the warps' outputs become the piece's
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int half = 0; half < 2; half++) {
        float x = l[mt][half];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (t4 == 0) {
          const int at = (mt * 16 + half * 8 + g) * A8_WARPS + warp;
          s_m[at] = m[mt][half];
          s_l[at] = x;
        }
      }
    }
    if (lane == 0) s_e[warp] = E;
    if (warp != 0) asm volatile("bar.sync 1, %0;" ::"n"(A8_THREADS) : "memory");
    const bool whole = p.pieces == 1;
    float* part = part8_at<D, ROWS>(a.part, me, p.lo == 0);
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
      if (mt * 16 >= p.rows) break;
      // a thread has columns (2 t4) * NT .. and (2 t4 + 1) * NT .., which are neighbours
#pragma unroll
      for (int half = 0; half < 2; half++) {
        float* dst = s_o + (warp * 16 + half * 8 + g) * L::O_ROW + t4 * L::O_GROUP;
#pragma unroll
        for (int side = 0; side < 2; side++)
#pragma unroll
          for (int j = 0; j < NT; j += 4)
            *reinterpret_cast<float4*>(dst + side * NT + j) =
                make_float4(o[mt][j][2 * half + side], o[mt][j + 1][2 * half + side], o[mt][j + 2][2 * half + side], o[mt][j + 3][2 * half + side]);
      }
      if (mt == 0 && nx.valid) start(nx);
      __syncthreads();
      int Emax = -1000;
#pragma unroll
      for (int w = 0; w < A8_WARPS; w++) Emax = max(Emax, s_e[w]);
      for (int x = tid; x < 16 * (D / 4); x += A8_THREADS) {
        const int rr = x / (D / 4), col = (x % (D / 4)) * 4, all = mt * 16 + rr;
        if (all >= p.rows) break;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < A8_WARPS; w++) top = fmaxf(top, s_m[all * A8_WARPS + w]);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < A8_WARPS; w++) {
          const float lw = s_l[all * A8_WARPS + w];
          if (lw == 0.f) continue;  // the warp saw nothing
          const float mw = s_m[all * A8_WARPS + w], f = top == mw || mw == -INFINITY ? 1.f : exp2_fast(mw - top);
          sum = fmaf(f, lw, sum);
          if (s_e[w] < -500) continue;
          const float fe = f * exp2_fast((float)max(s_e[w] - Emax, -200));
          const float4 z = *reinterpret_cast<const float4*>(s_o + (w * 16 + rr) * L::O_ROW + col / DIMS * L::O_GROUP + col % DIMS);
          y.x = fmaf(fe, z.x, y.x);
          y.y = fmaf(fe, z.y, y.y);
          y.z = fmaf(fe, z.z, y.z);
          y.w = fmaf(fe, z.w, y.w);
        }
        const bool none = sum == 0.f;
        const float inv = none ? 0.f : exp2f((float)max(Emax, -140)) / sum;
        y = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        const float log2sum = none ? -INFINITY : (top == -INFINITY ? 0.f : top - A8_UP) + log2f(sum);
        if (whole) {
          const int gr = p.row0 + all, tok = gr / a.group;
          const int64_t at = (int64_t)(p.t0 + tok) * a.hq + p.h * a.group + (gr - tok * a.group);
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + col) = make_uint2(pack2<T>(y.x, y.y), pack2<T>(y.z, y.w));
          if (a.lse && col == 0) a.lse[at] = log2sum * 0.69314718055994531f;
        } else {
          __stcg(reinterpret_cast<float4*>(part + all * D + col), y);
          if (col == 0) __stcg(part + ROWS * D + all, log2sum);
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
        for (int x = tid; x < p.rows * (D / 4); x += A8_THREADS) {
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
            float up = top;
#pragma unroll
            for (int j = 0; j < 8; j++) up = fmaxf(up, e[j]);
            const float f = top == -INFINITY ? 0.f : exp2_fast(top - up);
            sum *= f;
            y.x *= f; y.y *= f; y.z *= f; y.w *= f;
            top = up;
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
          const int gr = p.row0 + rr, tok = gr / a.group;
          const int64_t at = (int64_t)(p.t0 + tok) * a.hq + p.h * a.group + (gr - tok * a.group);
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + col) =
              make_uint2(pack2<T>(y.x * inv, y.y * inv), pack2<T>(y.z * inv, y.w * inv));
          if (a.lse && col == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        }
      }
      __syncthreads();  // s_last has been read
    } else if (MT > 1) {
      __syncthreads();  // the queries are there
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

template <class T, int D, int MT, bool WIN>
static cudaError_t attend8_launch(const AttendArgs& a, const tk_kv_cache* cache, cudaStream_t st) {
  constexpr int bytes = Attend8Shape<D, MT>::TOTAL;
  static bool set[64];  // by device
  if (cache->device >= 64 || !set[cache->device]) {
    const cudaError_t e = cudaFuncSetAttribute(k_kv_attend8<T, D, MT, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (cache->device < 64) set[cache->device] = true;
  }
  k_kv_attend8<T, D, MT, WIN><<<cache->sms, A8_THREADS, bytes, st>>>(a, cache->map_k, cache->map_v);
  return cudaGetLastError();
}

template <class T, int D, bool WIN>
static cudaError_t attend8_rows(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, cudaStream_t st) {
  return rows <= 16 ? attend8_launch<T, D, 1, WIN>(a, cache, st) : attend8_launch<T, D, 2, WIN>(a, cache, st);
}

template <class T, int D>
static cudaError_t attend8_pick(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, cudaStream_t st) {
  return a.window < INT32_MAX ? attend8_rows<T, D, true>(a, cache, rows, st) : attend8_rows<T, D, false>(a, cache, rows, st);
}

cudaError_t attend8(const AttendArgs& a, const tk_kv_cache* cache, int64_t rows, int grid, cudaStream_t st) {
  if (rows > 32) return attend8_many(a, cache, rows, grid, st);
  if (cache->type == TK_BF16)
    return cache->head_dim == 64 ? attend8_pick<__nv_bfloat16, 64>(a, cache, rows, st) : attend8_pick<__nv_bfloat16, 128>(a, cache, rows, st);
  return cache->head_dim == 64 ? attend8_pick<__half, 64>(a, cache, rows, st) : attend8_pick<__half, 128>(a, cache, rows, st);
}

}  // namespace tk
