// tk_kv.cu -- placing requests in a paged key/value cache (tk_kv_plan) and
// storing their rows there (tk_kv_append).
#include <algorithm>
#include <new>

#include "tk_blackwell.cuh"
#include "tk_kv.cuh"

namespace tk {

// ---------------------------------------------------------------- tk_kv_plan

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_ITEMS = 4;  // tokens per thread and step: one 16-byte store of positions

struct PlanArgs {
  const int64_t* off;
  const int32_t* ctx;
  int64_t R, T;
  int log2_bs;
  int32_t* table;
  int64_t table_stride, table_width;
  const int32_t* free_ids;
  int64_t n_free;
  const int64_t* cursor;
  const int32_t* parent;
  int32_t* pos;
  int64_t* slot;
  int32_t* req;
  int32_t* len;
  int64_t* mask;
  int64_t* info;
  int64_t per_cta;  // tokens of one CTA, a multiple of PLAN_ITEMS
};

// What a request with the offsets [o, e) asks of the free list: blocks, or -1 if
// it cannot be placed whatever the list holds.  Nothing is added before it is known to fit.
__device__ __forceinline__ int plan_need(const PlanArgs& a, int64_t o, int64_t e, int ctx) {
  if (o < 0 || e < o || e > a.T || ctx < 0 || e - o > INT32_MAX - 128 - ctx || (a.parent && e - o > KV_TREE_MAX)) return -1;
  const int up = (1 << a.log2_bs) - 1, want = (ctx + (int)(e - o) + up) >> a.log2_bs;
  return want > a.table_width ? -1 : want - ((ctx + up) >> a.log2_bs);
}

// Exclusive prefix of x over the block's threads; *total = the sum.
__device__ __forceinline__ int64_t plan_scan(int64_t x, int64_t* s_warp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // s_warp of an earlier call has been read
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int64_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < PLAN_THREADS / 32; w++) {
    const int64_t v = s_warp[w];
    if (w < warp) before += v;
    sum += v;
  }
  *total = sum;
  return before + incl - x;
}

// Request r takes the free blocks [cursor + sum of the needs before it, + its
// own), so every CTA finds its requests' blocks from the lengths alone: CTA c
// writes the tokens [c * per_cta, +per_cta), after adding up the needs of the
// requests before them (20 bytes a request, from L2).  No CTA waits for another and one
// launch does it all.  A new block's table entry is written by the token at its
// first place.  The last CTA writes the lengths and the totals.  The CTAs agree only if
// the offsets do not decrease, so each looks at all of them and places nothing otherwise.  A thread has four
// tokens and looks a block up where it begins: 5.3 M tokens of 4,096 prompts, bound by
// instructions at first (37 us), take 24 us; the 85 MB of outputs alone take 13 us.
__global__ void __launch_bounds__(PLAN_THREADS) k_kv_plan(PlanArgs a) {
  __shared__ int64_t s_warp[PLAN_THREADS / 32];
  __shared__ int s_off[PLAN_THREADS + 1];  // from t0 on
  __shared__ int s_base[PLAN_THREADS];     // free_ids index of the request's block 0 (new ones from `have` on)
  __shared__ int s_ctx[PLAN_THREADS];
  __shared__ bool s_placed[PLAN_THREADS];
  __shared__ int64_t s_first;
  const int tid = threadIdx.x, up = (1 << a.log2_bs) - 1;
  const int64_t cursor = a.cursor ? min(max(*a.cursor, (int64_t)0), a.n_free) : 0;

  if (blockIdx.x == gridDim.x - 1) {
    const int64_t per = (a.R + PLAN_THREADS - 1) / PLAN_THREADS;
    const int64_t r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
    int64_t sum = 0;
    bool bad = false;
#pragma unroll 4
    for (int64_t r = r0; r < r1; r++) {
      const int64_t o = a.off[r], e = a.off[r + 1];
      bad |= o < 0 || e < o;
      sum += max(plan_need(a, o, e, a.ctx[r]), 0);
    }
    const bool none = __syncthreads_or(bad);
    int64_t asked, taken, end = cursor + plan_scan(none ? 0 : sum, s_warp, &asked);
    int64_t took = 0, first = INT64_MAX;
#pragma unroll 4
    for (int64_t r = r0; r < r1; r++) {
      const int64_t o = a.off[r], e = a.off[r + 1];
      const int ctx = a.ctx[r], need = plan_need(a, o, e, ctx);
      if (need > 0) end += need;
      const bool placed = !none && (need == 0 || (need > 0 && end <= a.n_free));
      if (placed) took += need;
      else if (first == INT64_MAX && (!none || o < 0 || e < o)) first = r;
      a.len[r] = placed ? ctx + (int)(e - o) : ctx;
    }
    plan_scan(took, s_warp, &taken);
    if (tid == 0) s_first = INT64_MAX;
    __syncthreads();
    if (first != INT64_MAX) atomicMin((long long*)&s_first, (long long)first);
    __syncthreads();
    if (tid == 0) {
      const int64_t r = s_first;
      a.info[0] = cursor + taken;
      a.info[1] = asked;
      a.info[2] = r == INT64_MAX ? TK_OK
                  : plan_need(a, a.off[r], a.off[r + 1], a.ctx[r]) < 0 ? TK_E_LIMIT : TK_E_CAPACITY;
      a.info[3] = r == INT64_MAX ? -1 : r;
    }
    return;
  }

  const int64_t t0 = (int64_t)blockIdx.x * a.per_cta;
  const int count = (int)min(a.T - t0, a.per_cta);  // tokens of this CTA
  // the requests that end at or before t0: how many, and what they need
  int64_t skip = 0, sum = 0;
  bool bad = false;
#pragma unroll 4
  for (int64_t r = tid; r < a.R; r += PLAN_THREADS) {
    const int64_t o = a.off[r], e = a.off[r + 1];
    const int need = plan_need(a, o, e, a.ctx[r]);
    bad |= o < 0 || e < o;
    if (e <= t0) {
      skip++;
      sum += max(need, 0);
    }
  }
  int64_t r0, used;
  plan_scan(skip, s_warp, &r0);
  plan_scan(sum, s_warp, &used);
  if (__syncthreads_or(bad)) r0 = a.R;

  auto nobody = [&](int from, int to) {  // tokens of no request
    for (int t = from + tid; t < to; t += PLAN_THREADS) {
      const int64_t at = t0 + t;
      a.pos[at] = 0;
      a.req[at] = -1;
      a.slot[at] = -1;
      if (a.parent) a.mask[at] = 0;
    }
  };
  int lo = 0;  // tokens before lo are written
  if (r0 == 0 && a.R > 0) {  // what comes before the first request
    lo = (int)min((int64_t)count, max((int64_t)0, a.off[0] - t0));
    nobody(0, lo);
  }
  while (lo < count && r0 < a.R) {
    const int nr = (int)min((int64_t)PLAN_THREADS, a.R - r0);
    int need = 0;
    int64_t total;
    if (tid < nr) {
      const int64_t o = a.off[r0 + tid], e = a.off[r0 + tid + 1];
      const int ctx = a.ctx[r0 + tid];
      need = plan_need(a, o, e, ctx);
      s_off[tid] = (int)(min(o, a.T) - t0);
      s_ctx[tid] = ctx;
      if (tid == nr - 1) s_off[nr] = (int)(min(e, a.T) - t0);
    }
    const int64_t base = cursor + used + plan_scan(max(need, 0), s_warp, &total);
    if (tid < nr) {
      s_placed[tid] = need == 0 || (need > 0 && base + need <= a.n_free);
      s_base[tid] = (int)base - ((s_ctx[tid] + up) >> a.log2_bs);  // in range where it is used
    }
    // the requests that begin in this CTA's tokens: the search below is among them
    const int in = max(1, __syncthreads_count(tid < nr && s_off[tid] < count));
    const int hi = min(count, s_off[nr]);
    for (int g = (lo & ~(PLAN_ITEMS - 1)) + tid * PLAN_ITEMS; g < hi; g += PLAN_THREADS * PLAN_ITEMS) {
      int pos[PLAN_ITEMS], req[PLAN_ITEMS];
      int64_t slot[PLAN_ITEMS], mask[PLAN_ITEMS];
      // the request of the first token: the last that starts at or before it
      const int from = max(g, lo);
      int k = 0;
      for (int b = in; b > 1;) {
        const int h = b >> 1;
        if (s_off[k + h] <= from) k += h;
        b -= h;
      }
      const bool whole = g >= lo && g + PLAN_ITEMS <= hi;
      // of request k: spot = t + shift; its slots are first + (spot & within), first changes with the block
      int start, next, shift, within, blk;
      int64_t first;
      auto enter = [&]() {
        start = s_off[k];
        next = k + 1 < nr ? s_off[k + 1] : hi;  // the last one's tokens end the step
        shift = (int)((unsigned)s_ctx[k] - (unsigned)start);
        within = s_placed[k] ? up : 0;
        blk = s_placed[k] ? -1 : INT32_MAX;  // not placed: no block is looked up
        first = -1;
      };
      enter();
      if (whole && g >= start && g + PLAN_ITEMS <= next && within && !a.parent) {
        // nearly always: the four are one placed request's and lie in one block or two (looked up
        // in turn they took 26 us instead of 23 for 5.3 M tokens)
        const int c = s_ctx[k], have = (c + up) >> a.log2_bs, s0 = g + shift, b0 = s0 >> a.log2_bs,
                  b1 = (s0 + PLAN_ITEMS - 1) >> a.log2_bs;
        int32_t* row = a.table + (r0 + k) * a.table_stride;
        const int32_t* fresh = a.free_ids + s_base[k];
        const int id0 = b0 < have ? row[b0] : fresh[b0], id1 = b1 < have ? row[b1] : fresh[b1];
        if ((s0 & up) == 0 && b0 >= have) row[b0] = id0;
        if (b1 != b0 && b1 >= have) row[b1] = id1;
#pragma unroll
        for (int j = 0; j < PLAN_ITEMS; j++)
          slot[j] = (int64_t)((s0 + j) >> a.log2_bs == b0 ? id0 : id1) * (up + 1) + ((s0 + j) & up);
        const int64_t at = t0 + g;
        const int q = (int)r0 + k;
        *reinterpret_cast<int4*>(a.pos + at) = make_int4(s0, s0 + 1, s0 + 2, s0 + 3);
        *reinterpret_cast<int4*>(a.req + at) = make_int4(q, q, q, q);
        *reinterpret_cast<longlong2*>(a.slot + at) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(a.slot + at + 2) = make_longlong2(slot[2], slot[3]);
        continue;
      }
#pragma unroll
      for (int j = 0; j < PLAN_ITEMS; j++) {
        const int t = g + j;
        if (!whole && (t < lo || t >= hi)) continue;
        while (t >= next && k + 1 < nr) {
          k++;
          enter();
        }
        const int spot = (int)((unsigned)t + (unsigned)shift);
        if (blk != INT32_MAX && blk != spot >> a.log2_bs) {
          blk = spot >> a.log2_bs;
          const int c = s_ctx[k];
          int32_t* entry = a.table + (r0 + k) * a.table_stride + blk;
          int id = -1;
          if (t < start || blk >= a.table_width) {
            id = -1;  // of no request's tokens
          } else if (blk < (c + up) >> a.log2_bs) {
            id = *entry;
          } else if ((unsigned)(s_base[k] + blk) < (uint64_t)a.n_free) {
            id = a.free_ids[s_base[k] + blk];
            if ((spot & up) == 0) *entry = id;
          }
          first = (int64_t)id * (up + 1);
        }
        req[j] = (int)r0 + k;
        pos[j] = spot;
        slot[j] = first + (spot & within);
        if (a.parent) {
          const int i = t - start;
          uint64_t m = 0;
          int depth = 0;
          if (i >= 0 && i < KV_TREE_MAX) {
            const int32_t* parent = a.parent + t0 + start;
            int at = i;
            m = 1ull << at;
            for (int p = parent[i]; p >= 0 && p < at; p = parent[p]) {
              m |= 1ull << p;
              at = p;
              depth++;
            }
          }
          mask[j] = (int64_t)m;
          pos[j] = s_ctx[k] + depth;
        }
      }
      const int64_t at = t0 + g;
      if (whole) {
        *reinterpret_cast<int4*>(a.pos + at) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(a.req + at) = make_int4(req[0], req[1], req[2], req[3]);
        *reinterpret_cast<longlong2*>(a.slot + at) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(a.slot + at + 2) = make_longlong2(slot[2], slot[3]);
        if (a.parent) {
          *reinterpret_cast<longlong2*>(a.mask + at) = make_longlong2(mask[0], mask[1]);
          *reinterpret_cast<longlong2*>(a.mask + at + 2) = make_longlong2(mask[2], mask[3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < PLAN_ITEMS; j++) {
          if (g + j < lo || g + j >= hi) continue;
          a.pos[at + j] = pos[j];
          a.req[at + j] = req[j];
          a.slot[at + j] = slot[j];
          if (a.parent) a.mask[at + j] = mask[j];
        }
      }
    }
    lo = max(lo, hi);
    used += total;
    r0 += nr;
    __syncthreads();  // the batch's shared arrays have been read
  }
  nobody(lo, count);
}

// -------------------------------------------------------------- tk_kv_append

constexpr int APPEND_THREADS = 128;
constexpr int APPEND_FLIGHT = 8;  // passes of a warp in flight, 1 KB each

struct AppendArgs {
  const void* qkv;
  int64_t row_stride, T;
  int hq, hk, dim;
  const float* q_gain;
  const float* k_gain;
  float eps;
  const float* rope;
  int64_t rope_len;
  int rot;
  const int32_t* pos;
  const int64_t* slot;
  void* q;
  void* k;
  void* v;
  int64_t s_block, s_head, s_token, n_slots;
  int log2_bs;
  int chunks, passes;  // warps per token, passes of each
};

// y = x * rsqrt(mean(x^2) + eps) * gain for every head of queries and keys, then
// (a, b) -> (a cos - b sin, b cos + a sin); values are copied.
// Bound by the rows' bytes, so the arithmetic has to stay under them: LANES lanes
// hold a head, 16 elements each, as 8 pairs that rotate together (so that no element crosses
// lanes), and work on two of them per instruction; gain and rotation become
// four factors per pair, computed once per token and side.  A pass is 32 / LANES heads of one token;
// the passes of a warp arrive ahead in shared memory, each lane's elements in its own place
// (in registers, two passes ahead, 32,768 rows of 48 heads took 163 us instead of 140).
template <class T, int LANES, bool NEIGHBOURS>
__global__ void __launch_bounds__(APPEND_THREADS, 5) k_kv_append(AppendArgs a) {
  using P = Pair<T>;
  using T2 = typename P::type;
  constexpr int HEADS = 32 / LANES;
  __shared__ uint4 s_x[APPEND_THREADS / 32][APPEND_FLIGHT][2][32];
  const int lane = threadIdx.x & 31, l = lane % LANES, g = lane / LANES;
  const int64_t w = ((int64_t)blockIdx.x * APPEND_THREADS + threadIdx.x) >> 5;
  const int64_t t = w / a.chunks;
  if (t >= a.T) return;
  // the lane's two runs of 8 elements: pairs are (e0 + i, e1 + i), or neighbours in each
  const int half = a.rot >> 1;
  const bool rotated = l * 16 < a.rot, in_dim = l * 16 < a.dim;
  const bool apart = !NEIGHBOURS && rotated;
  const int e0 = apart ? l * 8 : l * 16, e1 = apart ? e0 + half : e0 + 8;
  const int turned = a.hq + a.hk, all = turned + a.hk;
  const int first = (int)(w - t * a.chunks) * a.passes, last = min(first + a.passes, (all + HEADS - 1) / HEADS);

  uint4(*mine)[2][32] = s_x[threadIdx.x >> 5];
  const T* src = static_cast<const T*>(a.qkv) + t * a.row_stride + (first * HEADS + g) * a.dim;
  auto fetch = [&](int p) {
    if (p < last && in_dim && p * HEADS + g < all) {
      const uint32_t d = smem_addr(&mine[p % APPEND_FLIGHT][0][lane]);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src + e0) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + 512), "l"(src + e1) : "memory");
    }
    src += HEADS * a.dim;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < APPEND_FLIGHT; i++) fetch(first + i);

  float cs[8], sn[8];  // of the 8 pairs
  if (rotated) {
    const int64_t p = a.pos[t];
    const bool known = p >= 0 && p < a.rope_len;
    const float4* rope = reinterpret_cast<const float4*>(a.rope + ((known ? p : 0) * half + l * 8) * 2);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float4 f = __ldg(rope + j);
      const float nan = __int_as_float(0x7fffffff);
      cs[2 * j] = known ? f.x : nan;
      sn[2 * j] = known ? f.y : nan;
      cs[2 * j + 1] = known ? f.z : nan;
      sn[2 * j + 1] = known ? f.w : nan;
    }
  }
  const int64_t slot = a.slot[t];
  const bool stored = slot >= 0 && slot < a.n_slots;
  const int64_t place = (slot >> a.log2_bs) * a.s_block + (slot & ((1 << a.log2_bs) - 1)) * a.s_token;

  // (x0, x1) -> (x0 f00 + x1 f01, x1 f11 + x0 f10), two pairs a register
  uint64_t f00[4], f01[4], f10[4], f11[4];
  int kind = -1;  // 0 queries, 1 keys, 2 values; of the lane's head
#pragma unroll 1
  for (int p = first; p < last; p++) {
    const int h = p * HEADS + g, k = h < a.hq ? 0 : h < turned ? 1 : 2;
    if (k != kind) {
      kind = k;
      const float* gain = k == 0 ? a.q_gain : a.k_gain;
      float g0[8], g1[8];
#pragma unroll
      for (int j = 0; j < 8; j++) g0[j] = g1[j] = 1.f;
      if (gain && in_dim && k < 2) {
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(gain + e0) + j), y = __ldg(reinterpret_cast<const float4*>(gain + e1) + j);
          g0[4 * j] = x.x; g0[4 * j + 1] = x.y; g0[4 * j + 2] = x.z; g0[4 * j + 3] = x.w;
          g1[4 * j] = y.x; g1[4 * j + 1] = y.y; g1[4 * j + 2] = y.z; g1[4 * j + 3] = y.w;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (!rotated) {
          f00[j] = pair64(g0[2 * j], g0[2 * j + 1]);
          f11[j] = pair64(g1[2 * j], g1[2 * j + 1]);
        } else if (NEIGHBOURS) {
          // registers are the pairs themselves: run 0 has pairs 0-3, run 1 pairs 4-7; the second
          // factors are for the neighbour
          f00[j] = pair64(g0[2 * j] * cs[j], g0[2 * j + 1] * cs[j]);
          f01[j] = pair64(-g0[2 * j + 1] * sn[j], g0[2 * j] * sn[j]);
          f11[j] = pair64(g1[2 * j] * cs[4 + j], g1[2 * j + 1] * cs[4 + j]);
          f10[j] = pair64(-g1[2 * j + 1] * sn[4 + j], g1[2 * j] * sn[4 + j]);
        } else {
          f00[j] = pair64(g0[2 * j] * cs[2 * j], g0[2 * j + 1] * cs[2 * j + 1]);
          f01[j] = pair64(-g1[2 * j] * sn[2 * j], -g1[2 * j + 1] * sn[2 * j + 1]);
          f11[j] = pair64(g1[2 * j] * cs[2 * j], g1[2 * j + 1] * cs[2 * j + 1]);
          f10[j] = pair64(g0[2 * j] * sn[2 * j], g0[2 * j + 1] * sn[2 * j + 1]);
        }
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(APPEND_FLIGHT - 1) : "memory");
    union Vec {
      uint4 u;
      T2 p[4];
    } x0, x1;
    x0.u = mine[p % APPEND_FLIGHT][0][lane];
    x1.u = mine[p % APPEND_FLIGHT][1][lane];
    fetch(p + APPEND_FLIGHT);
    if (p * HEADS < turned) {
      const bool normed = (k == 0 ? a.q_gain : a.k_gain) != nullptr;
      uint64_t y0[4], y1[4], ss = 0, ss2 = 0;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float2 u = P::up(x0.p[j]), v = P::up(x1.p[j]);
        y0[j] = pair64(u.x, u.y);
        y1[j] = pair64(v.x, v.y);
        ss = fma2(y0[j], y0[j], ss);
        ss2 = fma2(y1[j], y1[j], ss2);
      }
      const float2 s2 = unpair64(add2(ss, ss2));
      float s = in_dim ? s2.x + s2.y : 0.f;
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float inv = normed ? rsqrtf(s / (float)a.dim + a.eps) : 1.f;
      const uint64_t inv2 = pair64(inv, inv);
      if (k < 2) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          y0[j] = mul2(y0[j], inv2);
          y1[j] = mul2(y1[j], inv2);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
          uint64_t z0 = mul2(y0[j], f00[j]), z1 = mul2(y1[j], f11[j]);
          if (rotated) {
            if (NEIGHBOURS) {
              const float2 u = unpair64(y0[j]), v = unpair64(y1[j]);
              z0 = fma2(pair64(u.y, u.x), f01[j], z0);
              z1 = fma2(pair64(v.y, v.x), f10[j], z1);
            } else {
              z0 = fma2(y1[j], f01[j], z0);
              z1 = fma2(y0[j], f10[j], z1);
            }
          }
          const float2 u = unpair64(z0), v = unpair64(z1);
          x0.p[j] = P::down(u.x, u.y);
          x1.p[j] = P::down(v.x, v.y);
        }
      }
    }
    if (in_dim && h < all && (k == 0 || stored)) {
      T* dst = k == 0 ? static_cast<T*>(a.q) + (t * a.hq + h) * a.dim
                      : k == 1 ? static_cast<T*>(a.k) + place + (h - a.hq) * a.s_head
                               : static_cast<T*>(a.v) + place + (h - turned) * a.s_head;
      *reinterpret_cast<uint4*>(dst + e0) = x0.u;
      *reinterpret_cast<uint4*>(dst + e1) = x1.u;
    }
  }
}

template <class T, int LANES>
static void append_launch(AppendArgs& a, bool neighbours, int sms, cudaStream_t st) {
  constexpr int HEADS = 32 / LANES;
  const int all = (a.hq + 2 * a.hk + HEADS - 1) / HEADS;
  // a warp takes a token, or less of it while that fills the GPU's SMs with 16 warps each
  const int64_t enough = (int64_t)sms * 16;
  a.chunks = (int)std::min<int64_t>(all, std::max<int64_t>(1, enough / std::max<int64_t>(a.T, 1)));
  a.passes = (all + a.chunks - 1) / a.chunks;
  a.chunks = (all + a.passes - 1) / a.passes;
  const unsigned grid = (unsigned)((a.T * a.chunks * 32 + APPEND_THREADS - 1) / APPEND_THREADS);
  if (neighbours) k_kv_append<T, LANES, true><<<grid, APPEND_THREADS, 0, st>>>(a);
  else k_kv_append<T, LANES, false><<<grid, APPEND_THREADS, 0, st>>>(a);
}

template <class T>
static void append_lanes(AppendArgs& a, bool neighbours, int sms, cudaStream_t st) {
  if (a.dim <= 64) append_launch<T, 4>(a, neighbours, sms, st);
  else if (a.dim <= 128) append_launch<T, 8>(a, neighbours, sms, st);
  else append_launch<T, 16>(a, neighbours, sms, st);
}

}  // namespace tk

static int kv_arg(const char* where, const char* what) {
  tk_set_error("%s: %s", where, what);
  return TK_E_ARG;
}

static bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

extern "C" int tk_kv_plan(const int64_t* d_off, const int32_t* d_ctx, int64_t R, int64_t T, int block_size,
                          int32_t* d_table, int64_t table_stride, int64_t table_width,
                          const int32_t* d_free, int64_t n_free, const int64_t* d_cursor,
                          const int32_t* d_parent, int32_t* d_pos, int64_t* d_slot, int32_t* d_req,
                          int32_t* d_len, int64_t* d_mask, int64_t* d_info, void* cuda_stream) {
  using namespace tk;
  if (R < 0 || T < 0 || R >= INT32_MAX || T > INT32_MAX - 4096 || n_free < 0 || n_free > INT32_MAX || table_width < 0 ||
      table_stride < table_width)
    return kv_arg("tk_kv_plan", "bad size");
  if (!kv_block_size_ok(block_size)) return kv_arg("tk_kv_plan", "block_size is not a power of two from 16 to 128");
  if (!d_info || (R > 0 && (!d_off || !d_ctx || !d_len || (table_width > 0 && !d_table))) ||
      (T > 0 && (!d_pos || !d_slot || !d_req || (d_parent && !d_mask))) || (n_free > 0 && !d_free))
    return kv_arg("tk_kv_plan", "null pointer");
  if (!aligned16(d_pos) || !aligned16(d_slot) || !aligned16(d_req) || !aligned16(d_mask))
    return kv_arg("tk_kv_plan", "an output is not 16-byte aligned");
  // one CTA writes what another has yet to read
  const struct {
    const void* p;
    int64_t bytes;
  } ins[] = {{d_off, 8 * (R + 1)}, {d_ctx, 4 * R}, {d_free, 4 * n_free}, {d_cursor, 8}, {d_parent, 4 * T}},
    outs[] = {{d_pos, 4 * T}, {d_slot, 8 * T}, {d_req, 4 * T}, {d_len, 4 * R}, {d_mask, 8 * T}, {d_info, 32}};
  for (const auto& x : ins)
    for (const auto& y : outs)
      if (x.p && y.p && (uintptr_t)x.p < (uintptr_t)y.p + y.bytes && (uintptr_t)y.p < (uintptr_t)x.p + x.bytes)
        return kv_arg("tk_kv_plan", "an output overlaps an input");
  int dev = 0, sms = 1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    tk_set_error("tk_kv_plan: %s", cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  PlanArgs a = {d_off, d_ctx, R, T, kv_log2(block_size), d_table, table_stride, table_width, d_free, n_free,
                d_cursor, d_parent, d_pos, d_slot, d_req, d_len, d_mask, d_info, 0};
  // one step of every thread, or an even share of a few CTAs per SM
  const int64_t step = PLAN_THREADS * PLAN_ITEMS;
  const int64_t ctas = std::min<int64_t>((T + step - 1) / step, (int64_t)sms * 2);
  a.per_cta = ctas ? ((T + ctas - 1) / ctas + PLAN_ITEMS - 1) / PLAN_ITEMS * PLAN_ITEMS : 0;
  k_kv_plan<<<(unsigned)ctas + 1, PLAN_THREADS, 0, (cudaStream_t)cuda_stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) {
    tk_set_error("tk_kv_plan: %s", cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  return TK_OK;
}

// The cache as a tensor (element, token, head, block) whose box is 64
// elements of one head's block, or of half of one of 128 tokens: 128-byte rows, swizzled as the tensor cores read them.
static bool kv_map(const tk_kv_cache* c, void* mem, CUtensorMap* map) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return false;
  const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->block_size, (cuuint64_t)c->n_heads, (cuuint64_t)c->n_blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)c->stride[2] * 2, (cuuint64_t)c->stride[1] * 2, (cuuint64_t)c->stride[0] * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min(c->block_size, 64), 1, 1}, step[4] = {1, 1, 1, 1};
  return reinterpret_cast<Encode>(fn)(map, c->type == TK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                      4, mem, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

extern "C" int tk_kv_cache_create(void* d_k, void* d_v, int type, int64_t n_blocks, int n_heads, int block_size,
                                  int head_dim, const int64_t* stride, tk_kv_cache** out) {
  using namespace tk;
  const char* where = "tk_kv_cache_create";
  if (!out || !d_k || !d_v) return kv_arg(where, "null pointer");
  *out = nullptr;
  if (type != TK_BF16 && type != TK_F16) return kv_arg(where, "type is neither TK_BF16 nor TK_F16");
  if (n_blocks < 1 || n_blocks > INT32_MAX || n_heads < 1 || n_heads > 1024) return kv_arg(where, "bad size");
  if (!kv_block_size_ok(block_size)) return kv_arg(where, "block_size is not a power of two from 16 to 128");
  if (head_dim < 16 || head_dim > 256 || head_dim % 16) return kv_arg(where, "head_dim is not a multiple of 16 up to 256");
  int64_t st[3] = {(int64_t)n_heads * block_size * head_dim, (int64_t)block_size * head_dim, head_dim};
  for (int i = 0; i < 3 && stride; i++) {
    st[i] = stride[i];
    if (st[i] < head_dim || st[i] % 8 || st[i] >= (int64_t)1 << 38)
      return kv_arg(where, "a stride is below head_dim, no multiple of 8 elements, or 2^38 and more");
  }
  if (!aligned16(d_k) || !aligned16(d_v)) return kv_arg(where, "keys or values are not 16-byte aligned");
  int dev = 0, sms = 1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    tk_set_error("%s: %s", where, cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  tk_kv_cache* c = new (std::nothrow) tk_kv_cache();
  if (!c) {
    tk_set_error("%s: out of memory", where);
    return TK_E_NOMEM;
  }
  c->device = dev;
  c->sms = sms;
  c->type = type;
  c->n_blocks = n_blocks;
  c->n_heads = n_heads;
  c->block_size = block_size;
  c->log2_block = kv_log2(block_size);
  c->head_dim = head_dim;
  for (int i = 0; i < 3; i++) c->stride[i] = st[i];
  c->k = d_k;
  c->v = d_v;
  if (head_dim == 64 || head_dim == 128) {
    if (!kv_map(c, d_k, &c->map_k) || !kv_map(c, d_v, &c->map_v)) {
      delete c;
      tk_set_error("%s: the driver takes no tensor map of this layout", where);
      return TK_E_CUDA;
    }
  }
  *out = c;
  return TK_OK;
}

extern "C" void tk_kv_cache_free(tk_kv_cache* cache) { delete cache; }

extern "C" int tk_kv_append(const tk_kv_cache* cache, const void* d_qkv, int64_t row_stride, int64_t T, int n_q_heads,
                            const float* d_q_gain, const float* d_k_gain, float eps, const float* d_rope,
                            int64_t rope_len, int rot_dim, int neighbours, const int32_t* d_pos,
                            const int64_t* d_slot, void* d_q, void* cuda_stream) {
  using namespace tk;
  const char* where = "tk_kv_append";
  if (!cache) return kv_arg(where, "null cache");
  if (T < 0 || T > 1 << 26 || n_q_heads < 1 || n_q_heads > 1024 || rope_len < 0) return kv_arg(where, "bad size");
  if (row_stride < (int64_t)(n_q_heads + 2 * cache->n_heads) * cache->head_dim || row_stride % 8)
    return kv_arg(where, "row_stride is below a row's elements or no multiple of 8");
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16 || (rot_dim > 0 && !d_rope))
    return kv_arg(where, "rot_dim is not a multiple of 16 up to head_dim, or has no table");
  if (!(eps >= 0.f)) return kv_arg(where, "eps is negative");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != cache->device) return kv_arg(where, "the current device is not the cache's");
  if (T == 0) return TK_OK;
  if (!d_qkv || !d_slot || !d_q || (rot_dim > 0 && !d_pos)) return kv_arg(where, "null pointer");
  if (!aligned16(d_qkv) || !aligned16(d_q) || !aligned16(d_rope) || !aligned16(d_q_gain) || !aligned16(d_k_gain))
    return kv_arg(where, "a buffer is not 16-byte aligned");
  AppendArgs a = {d_qkv, row_stride, T, n_q_heads, cache->n_heads, cache->head_dim, d_q_gain, d_k_gain, eps, d_rope,
                  rope_len, rot_dim, d_pos, d_slot, d_q, cache->k, cache->v, cache->stride[0], cache->stride[1],
                  cache->stride[2], cache->n_blocks << cache->log2_block, cache->log2_block, 0, 0};
  if (cache->type == TK_BF16) append_lanes<__nv_bfloat16>(a, neighbours != 0, cache->sms, (cudaStream_t)cuda_stream);
  else append_lanes<__half>(a, neighbours != 0, cache->sms, (cudaStream_t)cuda_stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    tk_set_error("%s: %s", where, cudaGetErrorString(e));
    return TK_E_CUDA;
  }
  return TK_OK;
}
