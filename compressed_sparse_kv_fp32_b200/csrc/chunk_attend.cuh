// Causal attention of a ragged chunk of new tokens over the cache, on the tensor
// cores: one persistent kernel for one new token per sequence as for whole prompts.
//
// A unit is the work of one (sequence, kv head) and up to 2 x floor(128 / G) new
// tokens: their G query heads are the rows of two 128-row tiles, which share every
// K and V tile of 128 tokens.  Per tile: S = Q K^T (fp32, tensor memory), one running
// maximum and sum per row, P = exp2(s c - m) rounded to bf16 in tensor memory over S,
// O += P V (fp32, tensor memory).  The maximum that scales a row is raised only when a
// score exceeds it by more than kAtRaise, so O is hardly ever rescaled; the quotient is
// the same for every choice of it.
//
// P meets V, which is bf16, on the tensor cores, whose operands have one type; a product of
// P's lower bits would be a third one (512 cycles a tile beside 1024).  Its rounding, half a
// step of bf16 per probability and none in the sum they are divided by, is what the outputs
// lose besides their own: their error (root mean square over that of the outputs) is
// 0.0022-0.0023 over long caches, where the outputs' bf16 alone gives 0.0017.
//
// K and V tiles arrive by tensor-map copies of `box` rows -- all 128, or the largest
// power of two of at least 8 rows that divides the page size -- one lane per page piece;
// rows past the last visible slot are zeroed in V's tile (0 * NaN) and masked in S.  Page
// sizes without such a divisor are copied row by row with cp.async, at a fifth of the rate.
//
// Roles: warps 0-3 and 4-7 one row per thread of tile 0 and 1 (softmax, rescaling,
// epilogue); warps 8-9 copy Q and K rows, warps 10-11 V rows, through the block table;
// one thread of warp 12 issues the products.  While one tile's softmax runs, the other tile's products do.  A unit of
// one row tile (decode) takes its K/V tiles in turn as tile 0 and tile 1 -- the second
// copy of S and O would idle otherwise -- and merges the two states at its end.
//
// Work split.  All units make one line of K/V tiles that is cut into equal shares, one per
// block, so that every block does the same work whatever the lengths: a unit cut by a
// share's end leaves partial states in the workspace, and the block that arrives last
// merges them in the blocks' order.  On the line a sequence's heads whose K and V fit in
// L2 together are next to each other, so that the blocks at work on them at one time read
// K and V from L2.
// Products of one thread run in the order they were issued, which lets a tile's next S be
// made over its P; a barrier's answer and a commit are what costs between them.
//
// Bound by reading K and V for few rows (8 sequences of 16K-32K, one token each, 32 over 8
// heads: 145 us, 6.0 TB/s, 0.92 of the copy rate), and for many by the chain of one row
// tile -- softmax 1900 cycles, its two products 1024, handing over some 700 -- two of
// which share the tensor cores (2048 new tokens over 32K: 1.01 ms, 1050 TFLOP/s, 0.64 of
// the matrix rate; 0.53 under the power cap of a long run).  Tried: an issuing thread per
// row tile (the tiles fall into step: 1313 against 1087 us), halves of 64 tokens (1035
// against 980), a share of the exponentials as polynomials (none faster).
#pragma once

#include <cuda.h>

#include "chunk.cuh"
#include "umma.cuh"

namespace adamas {

constexpr int kAtThreads = 512;
constexpr int kAtStages = 2;  // of K, and of V
// A row's P is at most 2^16 and its sum and outputs at most 2^16 x 2^31 times a value: far
// inside the range of bf16 and fp32, whose precision does not depend on the scale; what
// underflows is 2^-110 of the largest and less.  (2^8: 1033 against 1012 us, 2048 new
// tokens over 32K.)
constexpr float kAtRaise = 16.0f;
constexpr int kAtMaxGrid = 160;
constexpr int kAtPartRow = 132;             // m, l, -, -, o[128]
constexpr int64_t kAtL2Bytes = 48ll << 20;  // K and V of heads that go through a wave together

// Where a block's share of the line begins, and how it goes on from there.
struct AtSeq {  // a sequence of the batch: its rows and length
  int first, n, len;
};
struct AtWalk {
  long long x, x1;  // [x, x1) of the line is still to do
  AtSeq sq;         // the sequence at x
  int hg;           // heads of its groups
  int b, group, q, h;  // sequence, group of heads, unit of the chunk, head in the group: the unit at x
  int t;               // x's place in the unit
};

// What a block keeps of the launch's plan, which it makes for itself (the lengths are on
// the device).
struct AtPlan {
  long long W;  // length of the line
  int shares;
  int cost;     // places of a unit's start
  AtWalk start;
};
// A unit's start and end cost about as much as two K/V tiles; where a block has fewer than
// four tiles, finer shares matter more and it counts as one (four sequences of one token
// over 1000: 18 us, with two 23; prompts of up to 4096 tokens: 475 us, with two 411).
constexpr int kAtUnitCost = 2, kAtCostTiles = 4;

// 32 rows of 128 bytes per softmax warp: rows pass through on their way out, so that a
// store covers whole lines
constexpr int kAtRowsOut = 32 * 128;
constexpr size_t kAtSmem = 2 * kTileBytes + 2 * kAtStages * kTileBytes + 8 * kAtRowsOut + 1024;
static_assert((kMaxBatch + 1) * sizeof(longlong2) <= 2 * kTileBytes, "the plan's table lies over the first tiles");

struct AtParams {
  ChunkParams c;
  float* part;        // [2 * grid][part_rows][kAtPartRow]
  uint32_t* arrived;  // [grid]
  int part_rows;
  int TQ;             // tokens of one 128-row tile
  int box;            // rows of a tensor-map copy; 0: rows are copied one by one
  int out_copies;     // a warp's 32 rows are whole tokens: they may leave by one copy
};

struct AtUnit {
  int b;                 // sequence
  int h, ntok;           // kv head, new tokens
  int row0;              // packed row of the first new token
  int pos0;              // slot of the first token (may be negative)
  int kv_end;            // slots that the last token sees
  int tiles;
};

struct AtSegment {
  AtUnit u;
  int t0, t1;      // K/V tiles [t0, t1) of the unit
  bool part;       // not the whole unit
  int slot, ca, cb;  // partial state's place; blocks that share the unit
};

__device__ __forceinline__ AtSeq at_seq(const AtParams& p, int b, bool& bad_cu, bool& bad_len) {
  AtSeq s;
  ragged_rows(p.c.cu_q, b, p.c.T, s.first, s.n, bad_cu);
  s.len = (int)clamp_len(p.c.seq_lens[b], p.c.geo.Nmax, bad_len);
  return s;
}
__device__ __forceinline__ AtSeq at_seq(const AtParams& p, int b) {
  bool bad = false;
  return at_seq(p, b, bad, bad);
}

__device__ __forceinline__ AtUnit at_unit(const AtParams& p, const AtSeq& sq, int b, int h, int qi) {
  AtUnit u;
  const int tu = 2 * p.TQ, tok0 = qi * tu;
  u.b = b;
  u.h = h;
  u.row0 = sq.first + tok0;
  u.ntok = sq.n - tok0 < tu ? sq.n - tok0 : tu;
  u.pos0 = sq.len - sq.n + tok0;
  const int end = u.pos0 + u.ntok;
  u.kv_end = end < 0 ? 0 : end;
  u.tiles = u.kv_end == 0 ? 1 : (u.kv_end + 127) / 128;
  return u;
}

// Units of a sequence per head, and the heads of a group: as many as have their K and V
// in L2 together.
__device__ __forceinline__ int at_units(const AtParams& p, const AtSeq& sq) {
  return (sq.n + 2 * p.TQ - 1) / (2 * p.TQ);
}
__device__ __forceinline__ int at_group(const AtParams& p, const AtSeq& sq) {
  const uint32_t fit = (uint32_t)(kAtL2Bytes / (4 * kDim)) / (uint32_t)(sq.len > 0 ? sq.len : 1);
  return fit < 1 ? 1 : (fit > (uint32_t)p.c.Hkv ? p.c.Hkv : (int)fit);
}

// a / b of two numbers that are nearly always below 2^32 (the long division takes 400 cycles).
__device__ __forceinline__ long long at_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The next piece of the block's share.  The line's order: sequences, groups of heads,
// units from the chunk's last tokens to its first, heads of the group; a unit takes
// pl.cost places and one per K/V tile.
__device__ __forceinline__ bool at_next(const AtPlan& pl, const AtParams& p, AtWalk& w, AtSegment& s) {
  while (w.x < w.x1) {
    const int hg = w.hg;
    s.u = at_unit(p, w.sq, w.b, w.group * hg + w.h, w.q);
    const long long f0 = w.x - w.t, f1 = f0 + pl.cost + s.u.tiles, e = w.x1 < f1 ? w.x1 : f1;
    s.t0 = w.t > pl.cost ? w.t - pl.cost : 0;
    s.t1 = (int)(e - f0) - pl.cost;
    s.part = s.t0 != 0 || e != f1;
    s.slot = 2 * (int)blockIdx.x + (s.t0 == 0 ? 1 : 0);
    if (s.part) {  // the blocks whose shares hold the unit's first and last tile
      s.ca = (int)at_div((f0 + pl.cost + 1) * pl.shares - 1, pl.W);
      s.cb = (int)at_div(f1 * pl.shares - 1, pl.W);
    }
    w.x = e;
    w.t = 0;
    if (e == f1 && w.x < w.x1 && ++w.h == (p.c.Hkv - w.group * hg < hg ? p.c.Hkv - w.group * hg : hg)) {
      w.h = 0;
      if (--w.q < 0) {
        ++w.group;
        if (w.group * hg >= p.c.Hkv) {
          w.group = 0;
          do w.sq = at_seq(p, ++w.b);  // the line goes on, so a sequence with rows follows
          while (w.sq.n == 0);
          w.hg = at_group(p, w.sq);
        }
        w.q = at_units(p, w.sq) - 1;
      }
    }
    if (s.t1 > s.t0) return true;  // else the share ends before the unit's first tile
  }
  return false;
}

// tab: shared memory for kMaxBatch + 1 numbers, free again afterwards.
__device__ __forceinline__ void at_make_plan(AtPlan& pl, const AtParams& p, longlong2* tab, int tid) {
  const int B = p.c.B, lane = tid & 31, warp = tid >> 5;
  for (int b = warp; b < B; b += kAtThreads / 32) {
    bool bad_cu = false, bad_len = false;
    const AtSeq sq = at_seq(p, b, bad_cu, bad_len);
    if (lane == 0 && bad_cu) atomicOr(p.c.err, kErrOffsets);
    if (lane == 0 && bad_len) atomicOr(p.c.err, kErrSeqLen);
    const int nu = at_units(p, sq);
    long long sum = 0;
    for (int q = lane; q < nu; q += 32) sum += at_unit(p, sq, b, 0, q).tiles;
    if (nu > 1) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    if (lane == 0) tab[b + 1] = make_longlong2(sum * p.c.Hkv, (long long)nu * p.c.Hkv);  // tiles, units
  }
  __syncthreads();
  if (warp == 0) {
    long long all = 0;
    for (int b = lane; b < B; b += 32) all += tab[b + 1].x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    const int cost = all >= (long long)kAtCostTiles * gridDim.x ? kAtUnitCost : 1;
    all = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      long long s = 0;
      if (b0 + lane < B) s = tab[b0 + lane + 1].x + cost * tab[b0 + lane + 1].y;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
      }
      s += all;
      if (b0 + lane < B) tab[b0 + lane + 1].x = s;  // from here on: places before the next sequence
      all = __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) tab[0].x = 0;
    __syncwarp();
    // a share is a unit's start and a tile at least
    const long long most = at_div(all, cost + 1);
    const int shares = most < (long long)gridDim.x ? (int)most : (int)gridDim.x;
    AtWalk w = {};
    if ((int)blockIdx.x < shares) {
      w.x = at_div(all * blockIdx.x, shares);
      w.x1 = at_div(all * (blockIdx.x + 1), shares);
      int lo = 0, hi = B;  // tab[lo] <= x < tab[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab[mid].x <= w.x) lo = mid;
        else hi = mid;
      }
      w.b = lo;
      const AtSeq sq = at_seq(p, lo);
      const int hg = at_group(p, sq), nu = at_units(p, sq);
      w.sq = sq;
      w.hg = hg;
      const long long per_head = at_div(tab[lo + 1].x - tab[lo].x, p.c.Hkv), y0 = w.x - tab[lo].x;
      w.group = (int)at_div(y0, per_head * hg);
      long long y = y0 - w.group * hg * per_head, before = 0;
      const int hc = p.c.Hkv - w.group * hg < hg ? p.c.Hkv - w.group * hg : hg;
      for (int k0 = 0; k0 < nu; k0 += 32) {
        const int places = k0 + lane < nu ? at_unit(p, sq, lo, 0, nu - 1 - k0 - lane).tiles + cost : 0;
        long long s = places;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long u = __shfl_up_sync(0xffffffffu, s, d);
          if (lane >= d) s += u;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, y < hc * (before + s));
        if (here) {
          const int l = __ffs(here) - 1;
          const int cl = __shfl_sync(0xffffffffu, places, l);
          y -= hc * (before + __shfl_sync(0xffffffffu, s, l) - cl);
          w.q = nu - 1 - k0 - l;
          w.h = (int)at_div(y, cl);
          w.t = (int)(y - (long long)w.h * cl);
          break;
        }
        before += __shfl_sync(0xffffffffu, s, 31);
      }
    }
    if (lane == 0) {
      pl.W = all;
      pl.shares = shares;
      pl.cost = cost;
      pl.start = w;
    }
    fence_async_smem();  // tensor-map copies write over the table next
  }
  __syncthreads();
}

// 32 rows of 128 bytes, one per lane in x, to their places (null: none): through shared
// memory, so that each store instruction covers four whole lines.
__device__ __forceinline__ void at_stage_rows(uint32_t buf, const uint32_t (&x)[32], int lane) {
#pragma unroll
  for (int c = 0; c < 8; ++c)  // in the 128-byte swizzle
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((c ^ (lane & 7)) << 4)), "r"(x[4 * c]),
                 "r"(x[4 * c + 1]), "r"(x[4 * c + 2]), "r"(x[4 * c + 3])
                 : "memory");
}
__device__ __forceinline__ void at_store_rows(uint32_t buf, const uint32_t (&x)[32], void* row, int lane) {
  at_stage_rows(buf, x, lane);
  __syncwarp();
  const uint64_t mine = reinterpret_cast<uint64_t>(row);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3), c = lane & 7;
    const uint64_t to = __shfl_sync(0xffffffffu, mine, r);
    const uint4 v = lds128(buf + r * 128 + ((c ^ (r & 7)) << 4));
    if (to) *reinterpret_cast<uint4*>(to + 16 * c) = v;
  }
  __syncwarp();
}

__global__ void __launch_bounds__(kAtThreads, 1)
    chunk_attend_kernel(const AtParams p, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap o_map) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ AtPlan pl;
  __shared__ __align__(8) uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], k_full[kAtStages],
      k_empty[kAtStages], v_full[kAtStages], v_empty[kAtStages], v_tail[kAtStages], all_done;
  __shared__ float2 duo[128];  // state of the second half of a one-tile unit
  __shared__ uint32_t tmem_slot, gave_up, last_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_tile = base, k_ring = base + 2 * kTileBytes, v_ring = k_ring + kAtStages * kTileBytes,
                 rows_out = v_ring + kAtStages * kTileBytes;

  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
    }
    for (int i = 0; i < kAtStages; ++i) {
      mbar_init(&k_full[i], 64);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 64);
      mbar_init(&v_empty[i], 1);
      mbar_init(&v_tail[i], 1);
    }
    mbar_init(&all_done, 1);
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc512(&tmem_slot);
  tmem_fence_before();
  at_make_plan(pl, p, reinterpret_cast<longlong2*>(smem_raw + (base - smem_addr(smem_raw))), tid);  // ends with a barrier
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;  // columns: S0 | S1 | O0 | O1, 128 each

  if (warp < 8) {
    // ------------------------------------------------------------ softmax and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int t = warp >> 2;                      // tile
    const int r = (warp & 3) * 32 + lane;         // row of the tile
    const uint32_t quad = (uint32_t)(warp & 3) << 21;  // 32 lanes, in the address's upper half
    const uint32_t S = tmem + quad + 128 * t, O = tmem + quad + 256 + 128 * t;
    const int G = p.c.G, rt = r / G, rg = r - rt * G;  // the row's token in the tile, its head in the group
    AtWalk w = pl.start;
    AtSegment sg;
    uint32_t s_par = 0, o_par = 0;
    while (at_next(pl, p, w, sg)) {
      const bool two = sg.u.ntok > p.TQ;           // two row tiles, or one whose K/V tiles alternate
      const int tok = two ? t * p.TQ + rt : rt;
      const int rows = (sg.u.ntok - (two ? t * p.TQ : 0)) * G;  // live rows of the tile (may be above 128)
      const int step = two ? 1 : 2, j0 = two ? sg.t0 : sg.t0 + t;
      if (j0 < sg.t1) {
        const bool live = rt < p.TQ && tok < sg.u.ntok;
        const bool warp_live = (warp & 3) * 32 < rows;
        const int vis = live ? (sg.u.pos0 + tok + 1 < 0 ? 0 : sg.u.pos0 + tok + 1) : 0;  // slots it sees
        // all rows of the warp see at least this many (dead rows aside)
        const int vis_all = __reduce_min_sync(0xffffffffu, live ? vis : 0x7fffffff);
        float m = -INFINITY, l = 0.0f;
        for (int j = j0; j < sg.t1; j += step) {
          mbar_wait_or_give_up(&s_full[t], s_par, &gave_up);
          s_par ^= 1;
          if (warp_live) {
            tmem_fence_after();
            uint32_t x[4][32];
            tmem_ld32(S, x[0]);
            tmem_ld32(S + 32, x[1]);
            tmem_ld32(S + 64, x[2]);
            tmem_ld32(S + 96, x[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_wait_ld(x[c]);
            if (j * 128 + 128 > vis_all) {  // some row does not see the whole tile
              const int seen = vis - j * 128;
#pragma unroll
              for (int i = 0; i < 128; ++i) x[i >> 5][i & 31] = i < seen ? x[i >> 5][i & 31] : 0xFF800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 128; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mx[k] = max3(mx[k], __uint_as_float(x[i >> 5][(i & 31) + k]), __uint_as_float(x[i >> 5][(i & 31) + 4 + k]));
            const float mt = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]) * kScoreLog2;
            const bool raise = mt > m + kAtRaise;  // also when m is -inf and a score is not
            if (__any_sync(0xffffffffu, raise)) {
              const float mn = raise ? mt : m;
              const float f = raise ? fast_exp2(m - mn) : 1.0f;  // 0 when m was -inf
              m = mn;
              l *= f;
              if (j > j0) {  // every product into O is done: S of this tile came after them
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(O + c, o);
                  tmem_wait_ld16(o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st16(O + c, o);
                }
              }
            }
            const float sub = m == -INFINITY ? 0.0f : m;
            const uint64_t scale2 = f2_pack(kScoreLog2, kScoreLog2), sub2 = f2_pack(-sub, -sub);
            uint64_t sum[2] = {0, 0};  // two pairs of fp32 sums
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t y[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint64_t e = f2_fma(f2_pack(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])), scale2, sub2);
                float a, b;
                f2_unpack(e, a, b);
                a = fast_exp2(a);
                b = fast_exp2(b);
                sum[i & 1] = f2_add(sum[i & 1], f2_pack(a, b));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y[i]) : "f"(b), "f"(a));
              }
              tmem_st16(S + 16 * c, y);  // over columns of S that were read
            }
            {
              float a, b;
              f2_unpack(f2_add(sum[0], sum[1]), a, b);
              l += a + b;
            }
            tmem_wait_st();
            tmem_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[t]);
        }
        // ---- epilogue
        mbar_wait_or_give_up(&o_full[t], o_par, &gave_up);
        o_par ^= 1;
        tmem_fence_after();
        const bool merge = !two && sg.t1 - sg.t0 > 1;
        float fa = 1.0f, fb = 0.0f;  // factors of this state and of the other one
        if (merge) {
          // tile 1's threads hand their maximum and sum to tile 0's, whose threads read both O
          if (t == 1) {
            duo[r] = make_float2(m, l);
            tmem_fence_before();
          }
          named_sync(2, 256);
          if (t == 0) {
            tmem_fence_after();
            const float2 other = duo[r];
            const float M = fmaxf(m, other.x);
            if (M != -INFINITY) {
              fa = fast_exp2(m - M);
              fb = fast_exp2(other.x - M);
              l = l * fa + other.y * fb;
              m = M;
            }
          }
        }
        if (warp_live && !(merge && t == 1)) {
          const int64_t row = (int64_t)(sg.u.row0 + tok) * p.c.Hq + sg.u.h * G + rg;
          float* st = p.part + ((int64_t)sg.slot * p.part_rows + (tok * G + rg)) * kAtPartRow;
          if (!sg.part) {
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;  // a row that sees nothing: O is 0 as well
            fa *= inv;
            fb *= inv;
          }
          const uint32_t buf = rows_out + warp * kAtRowsOut;
          const bool whole = p.out_copies && __all_sync(0xffffffffu, live);
          if (whole && !merge && !sg.part) {  // the common end of a prompt's unit, in as little code as it takes
            if (lane == 0) tma_store_wait_read();
            __syncwarp();
            const uint64_t f2 = f2_pack(fa, fa);
#pragma unroll 1
            for (int c0 = 0; c0 < 128; c0 += 64) {
              uint32_t x[32], z[32], y[32];
              tmem_ld32(O + c0, x);
              tmem_ld32(O + c0 + 32, z);
              tmem_wait_ld(x);
              tmem_wait_ld(z);
              const uint64_t zero = 0;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float a, b;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(i < 16 ? x[2 * i] : z[2 * i - 32]),
                                         __uint_as_float(i < 16 ? x[2 * i + 1] : z[2 * i - 31])), f2, zero), a, b);
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y[i]) : "f"(b), "f"(a));
              }
              if (c0) {
                if (lane == 0) tma_store_wait_read();
                __syncwarp();
              }
              at_stage_rows(buf, y, lane);
              fence_async_smem();
              __syncwarp();
              if (lane == 0) tma_store_3d(&o_map, c0, sg.u.h * G, sg.u.row0 + tok, buf);
            }
          } else
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 64) {
            uint32_t y[32];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int c = c0 + 32 * hf;
              uint32_t x[32];
              tmem_ld32(O + c, x);
              tmem_wait_ld(x);
              if (merge) {
                uint32_t z[32];
                tmem_ld32(O + 128 + c, z);
                tmem_wait_ld(z);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  x[i] = __float_as_uint(__uint_as_float(x[i]) * fa + __uint_as_float(z[i]) * fb);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * fa);
              }
              if (sg.part) {
                if (lane == 0) tma_store_wait_read();
                __syncwarp();
                at_store_rows(buf, x, live ? st + 4 + c : nullptr, lane);
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                      : "=r"(y[16 * hf + i])
                      : "f"(__uint_as_float(x[2 * i + 1])), "f"(__uint_as_float(x[2 * i])));
              }
            }
            if (!sg.part) {
              if (lane == 0) tma_store_wait_read();
              __syncwarp();
              at_store_rows(buf, y, live ? p.c.out + row * kDim + c0 : nullptr, lane);
            }
          }
          if (live) {
            if (sg.part) *reinterpret_cast<float2*>(st) = make_float2(m, l);
            else if (p.c.lse) p.c.lse[row] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
          }
        }
        tmem_fence_before();
        // tile 0 has read both O before tile 1 lets the next products into its own
        if (merge) named_sync(2, 256);
      }
      if (sg.part) {
        // the last of the unit's blocks to arrive merges the states, in the blocks' order
        __threadfence();
        named_sync(1, 256);
        if (tid == 0) {
          const uint32_t before = atomicAdd(&p.arrived[sg.ca], 1u);
          last_flag = before == (uint32_t)(sg.cb - sg.ca);
          if (last_flag) p.arrived[sg.ca] = 0;
        }
        named_sync(1, 256);
        if (last_flag) {
          __threadfence();
          // eight lanes a row, sixteen columns a lane, so that a warp has four rows' loads
          // under way; the states one after the other, each joined by its weight
          const int rows_all = sg.u.ntok * G;
          const int64_t state = (int64_t)2 * p.part_rows * kAtPartRow;  // from one block's to the next one's
          for (int pr = warp * 4 + (lane >> 3); pr < rows_all; pr += 32) {
            // the first block's state is in its second place
            const float* st = p.part + ((int64_t)(2 * sg.ca + 1) * p.part_rows + pr) * kAtPartRow;
            const float* next = p.part + ((int64_t)2 * sg.ca * p.part_rows + pr) * kAtPartRow + state;
            float M = -INFINITY, L = 0.0f;
            float o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = 0.0f;
#pragma unroll 5
            for (int c = sg.ca; c <= sg.cb; ++c) {
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(st));
              float4 x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = __ldcg(reinterpret_cast<const float4*>(st + 4) + (lane & 7) + 8 * i);
              st = next;
              next += state;
              const float Mn = fmaxf(M, ml.x), sub = Mn == -INFINITY ? 0.0f : Mn;
              const float f = fast_exp2(M - sub), g = fast_exp2(ml.x - sub);
              M = Mn;
              L = L * f + ml.y * g;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[4 * i] = o[4 * i] * f + x[i].x * g;
                o[4 * i + 1] = o[4 * i + 1] * f + x[i].y * g;
                o[4 * i + 2] = o[4 * i + 2] * f + x[i].z * g;
                o[4 * i + 3] = o[4 * i + 3] * f + x[i].w * g;
              }
            }
            const float inv = L > 0.0f ? 1.0f / L : 0.0f;
            const int tk = pr / G;
            const int64_t row = (int64_t)(sg.u.row0 + tk) * p.c.Hq + sg.u.h * G + (pr - tk * G);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t y0, y1;
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y0) : "f"(o[4 * i + 1] * inv), "f"(o[4 * i] * inv));
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y1) : "f"(o[4 * i + 3] * inv), "f"(o[4 * i + 2] * inv));
              reinterpret_cast<uint2*>(p.c.out + row * kDim)[(lane & 7) + 8 * i] = make_uint2(y0, y1);
            }
            if ((lane & 7) == 0 && p.c.lse) p.c.lse[row] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
          }
        }
        named_sync(1, 256);  // last_flag is read before the next unit sets it
      }
    }
    if (lane == 0) tma_store_wait();
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp < 12) {
      // ---------------------------------------------------------- copies
      const bool is_v = warp >= 10;
      const int lt = (tid - 256) & 63, lr = lt >> 4, lc = lt & 15;  // rows lr + 4 i, piece lc
      const uint32_t piece[2] = {tile_piece(lr, lc), tile_piece(lr + 4, lc)};  // then + 1024 every 8 rows
      const uint16_t* rows_of = (is_v ? p.c.V : p.c.K) + lc * 8;
      const uint32_t ring = is_v ? v_ring : k_ring;
      uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
      AtWalk w = pl.start;
      AtSegment sg;
      uint32_t it = 0, nseg = 0, tails = 0;  // bit i: parity of the phase of v_tail[i] that comes next
      bool bad = false;
      while (at_next(pl, p, w, sg)) {
        if (!is_v && lt == 0) {  // Q: TQ tokens' heads of the group are TQ * G rows of a tile
          mbar_wait_or_give_up(&q_empty, (nseg & 1) ^ 1, &gave_up);
          const int nt = sg.u.ntok > p.TQ ? 2 : 1, tok = sg.u.row0;
          mbar_arrive_expect_tx(&q_full, (uint32_t)(nt * p.TQ * p.c.G * 2 * kDim));
          for (int t = 0; t < nt; ++t) {
            tma_load_3d(q_tile + t * kTileBytes, &q_map, 0, sg.u.h * p.c.G, tok + t * p.TQ, &q_full);
            tma_load_3d(q_tile + t * kTileBytes + kTileHalf, &q_map, 64, sg.u.h * p.c.G, tok + t * p.TQ, &q_full);
          }
        }
        ++nseg;
        for (int j = sg.t0; j < sg.t1; ++j, ++it) {
          const int stage = it % kAtStages;
          const uint32_t dst = ring + stage * kTileBytes;
          const uint32_t par = ((it / kAtStages) & 1) ^ 1;
          if (p.box) {
            const int seen = sg.u.kv_end - j * 128;  // rows of the tile that some row sees
            const int pieces = seen <= 0 ? 0 : ((seen < 128 ? seen : 128) + p.box - 1) / p.box;
            uint32_t row = 0;
            if (lt < pieces) row = p.c.geo.row32(sg.u.b, sg.u.h, j * 128 + lt * p.box, bad);
            mbar_wait_or_give_up(&empty[stage], par, &gave_up);
            const bool zeros = is_v && seen < 128;
            // (a tail's barrier is the stage's own: it is armed again only once both warps have
            // arrived at full[stage], behind their wait for the phase before)
            uint64_t* bar = zeros ? &v_tail[stage] : &full[stage];
            if (lt == 0) mbar_arrive_expect_tx(bar, (uint32_t)(pieces * p.box * 2 * kDim));
            if (lt < 32) {
              __syncwarp();
              if (lt < pieces) {
                const void* map = is_v ? &v_map : &k_map;
                tma_load_2d(dst + lt * p.box * 128, map, 0, (int)row, bar);
                tma_load_2d(dst + kTileHalf + lt * p.box * 128, map, 64, (int)row, bar);
              }
            }
            if (zeros) {
              mbar_wait_or_give_up(bar, (tails >> stage) & 1, &gave_up);
              tails ^= 1u << stage;
              for (int r = (seen < 0 ? 0 : seen) + lr; r < 128; r += 4)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + tile_piece(r, lc)), "r"(0) : "memory");
              fence_async_smem();
            }
            if (lt != 0 || zeros) mbar_arrive(&full[stage]);
            continue;
          }
          const int tb = j * 128 + lr;
          mbar_wait_or_give_up(&empty[stage], par, &gave_up);
#pragma unroll 1
          for (int i0 = 0; i0 < 128; i0 += 32) {  // rows i0 + lr + 4 i
            uint32_t row[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int tk = tb + i0 + 4 * i;
              row[i] = tk < sg.u.kv_end ? p.c.geo.row32(sg.u.b, sg.u.h, tk, bad) : 0u;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              cp_async16_or_zero(dst + piece[i & 1] + 128 * i0 + 1024 * (i >> 1), rows_of + (int64_t)row[i] * kDim,
                                 tb + i0 + 4 * i < sg.u.kv_end);
          }
          cp_async_arrive(&full[stage]);
        }
      }
      cp_async_wait<0>();
      // the copies land before the block goes, also when somebody gave up waiting for them
      for (uint32_t k = 1; k <= kAtStages && k <= it; ++k)
        mbar_wait_timed(&full[(it - k) % kAtStages], ((it - k) / kAtStages) & 1, 1000000000ull);
      if (is_v)  // (a stage without a tail so far: the phase before its first one counts as over)
        for (int i = 0; i < kAtStages; ++i) mbar_wait_timed(&v_tail[i], ((tails >> i) & 1) ^ 1, 1000000000ull);
      if (!is_v && nseg > 0) mbar_wait_timed(&q_full, (nseg - 1) & 1, 1000000000ull);
      if (bad) atomicOr(p.c.err, kErrTable);
    } else if (warp == 12) {
      // ---------------------------------------------------------- products
      if (lane == 0) {
        AtWalk w = pl.start;
        AtSegment sg;
        uint32_t ik = 0, iv = 0, nseg = 0, p_par[2] = {0, 0};
        // K tile -> S of t for the row tiles of the unit (or its only one)
        auto scores = [&](int t, int qt) {
          mma_rows_rows(tmem + 128 * t, q_tile + qt * kTileBytes, k_ring + (ik % kAtStages) * kTileBytes);
          mma_commit(&s_full[t]);
        };
        auto k_wait = [&]() {
          mbar_wait_or_give_up(&k_full[ik % kAtStages], (ik / kAtStages) & 1, &gave_up);
          if (!p.box) fence_async_smem();
        };
        auto k_next = [&]() { mma_commit(&k_empty[ik++ % kAtStages]); };
        auto outputs = [&](int t, bool acc, bool known) {
          if (!known) mbar_wait_or_give_up(&p_full[t], p_par[t], &gave_up);
          p_par[t] ^= 1;
          tmem_fence_after();
          mma_probs_rows(tmem + 256 + 128 * t, tmem + 128 * t, v_ring + (iv % kAtStages) * kTileBytes, acc);
        };
        while (at_next(pl, p, w, sg)) {
          const bool two = sg.u.ntok > p.TQ;
          const int n = sg.t1 - sg.t0, ahead = two ? 1 : 2;  // K tiles whose scores are under way
          mbar_wait_or_give_up(&q_full, nseg & 1, &gave_up);
          ++nseg;
          for (int j = 0; j < ahead && j < n; ++j) {
            k_wait();
            tmem_fence_after();
            scores(two ? 0 : j, 0);
            if (two) scores(1, 1);
            k_next();
          }
          if (two) {
            // A question to a barrier takes some 150 cycles and a commit 90, in which the tensor
            // cores go through what was issued (about three products of sixteen columns) and then
            // idle; so the questions for the next products are asked, and the buffers of the last
            // ones given back, between two products of the same tile.
            bool v_in = mbar_try(&v_full[iv % kAtStages], (iv / kAtStages) & 1);
            bool k_in = n > 1 && mbar_try(&k_full[ik % kAtStages], (ik / kAtStages) & 1);
            for (int j = 0; j < n; ++j) {
              const bool more = j + 1 < n;
              if (!v_in) mbar_wait_or_give_up(&v_full[iv % kAtStages], (iv / kAtStages) & 1, &gave_up);
              if (more && !k_in) mbar_wait_or_give_up(&k_full[ik % kAtStages], (ik / kAtStages) & 1, &gave_up);
              if (!p.box) fence_async_smem();
              outputs(0, j > 0, false);
              if (j > 0) {  // the buffers of the tiles before (their products precede this one)
                mma_commit(&v_empty[(iv - 1) % kAtStages]);
                mma_commit(&k_empty[(ik - 1) % kAtStages]);
              }
              const bool p_in = mbar_try(&p_full[1], p_par[1]);
              if (more) scores(0, 0);
              else mma_commit(&o_full[0]);
              outputs(1, j > 0, p_in);
              if (more) {
                v_in = mbar_try(&v_full[(iv + 1) % kAtStages], ((iv + 1) / kAtStages) & 1);
                k_in = j + 2 < n && mbar_try(&k_full[(ik + 1) % kAtStages], ((ik + 1) / kAtStages) & 1);
                scores(1, 1);
                if (j + 2 == n) mma_commit(&q_empty);  // Q was read for the last time
                ++ik;
              } else {
                mma_commit(&o_full[1]);
                mma_commit(&v_empty[iv % kAtStages]);
              }
              ++iv;
            }
          } else {
            for (int j = 0; j < n; ++j) {
              const bool more = j + 2 < n;
              const int t = j & 1;
              const bool v_in = mbar_try(&v_full[iv % kAtStages], (iv / kAtStages) & 1);
              const bool p_in = mbar_try(&p_full[t], p_par[t]);
              if (!v_in) mbar_wait_or_give_up(&v_full[iv % kAtStages], (iv / kAtStages) & 1, &gave_up);
              if (!p.box) fence_async_smem();
              outputs(t, j > 1, p_in);
              mma_commit(&v_empty[iv++ % kAtStages]);
              if (more) {
                k_wait();
                scores(t, 0);
                k_next();
                if (j + 3 == n) mma_commit(&q_empty);
              } else {
                mma_commit(&o_full[t]);
              }
            }
          }
          if (n <= ahead) mma_commit(&q_empty);
        }
        mma_commit(&all_done);
        mbar_wait_or_give_up(&all_done, 0, &gave_up);
      }
      __syncwarp();
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 12) tmem_free512(tmem);
  if (tid == 0 && gave_up) atomicOr(p.c.err, kErrTimeout);
}

}  // namespace adamas
