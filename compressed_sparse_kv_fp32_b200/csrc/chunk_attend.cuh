// Causal attention of a ragged chunk of new tokens over the cache, on the tensor
// cores: one persistent kernel for one new token per sequence as for whole prompts.
//
// A unit is the work of one (sequence, kv head) and up to 2 x floor(128 / G) new
// tokens: their G query heads are the rows of two 128-row tiles, which share every
// K and V tile of 128 tokens.  Per tile: S = Q K^T (fp32, tensor memory), one running
// maximum and sum per row, P = exp2(s c - m) rounded to bf16 in tensor memory over S,
// O += P V (fp32, tensor memory).  The maximum that scales a row is raised only when a
// score exceeds it by more than 2^8 in the exponent, so O is hardly ever rescaled; the
// quotient is the same for every choice of it, and P and the sum stay far from fp32's
// and bf16's range.
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
// Work split.  Sequences with several units (prompts) fill whole waves of the grid,
// heads that fit in L2 together next to each other and the longest units first, so that
// the blocks of a wave read the same K and V tiles at about the same time.  What is left
// over, and every sequence with a single unit (decode), is one line of K/V tiles cut
// into equal shares, one per block: a unit cut by a share's end leaves partial states
// in the workspace, and the block that arrives last merges them in the units' order.
#pragma once

#include <cuda.h>

#include "chunk.cuh"
#include "umma.cuh"

namespace adamas {

constexpr int kAtThreads = 512;
constexpr int kAtStages = 2;  // of K, and of V
constexpr int kAtMaxGrid = 160;
constexpr int kAtPartRow = 132;             // m, l, -, -, o[128]
constexpr int64_t kAtL2Bytes = 48ll << 20;  // K and V of heads that go through a wave together

// Plan of a launch, made by every block for itself (the lengths are on the device).
struct AtPlan {
  int mpre[kMaxBatch + 1];            // units of the sequences with several, before each
  long long spre[kMaxBatch + 1];      // tiles of the sequences with one unit per head, before each
  long long lpre[kAtMaxGrid + 1];            // tiles of the left-over units, before each
  int first[kMaxBatch];               // the sequence's rows
  int n[kMaxBatch];
  int len[kMaxBatch];
  long long W, Wl;   // tiles of the line, of its left-over units
  int waves, left, shares;
};

constexpr size_t kAtSmem = 2 * kTileBytes + 2 * kAtStages * kTileBytes + 1024;

struct AtParams {
  ChunkParams c;
  float* part;        // [2 * grid][part_rows][kAtPartRow]
  uint32_t* arrived;  // [grid]
  int part_rows;
  int TQ;             // tokens of one 128-row tile
  int box;            // rows of a tensor-map copy; 0: rows are copied one by one
};

struct AtUnit {
  int b, h, tok0, ntok;  // sequence, kv head, first new token, new tokens
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

struct AtWalk {
  int wave = 0;
  long long x, x1;
};

__device__ __forceinline__ AtUnit at_unit(const AtPlan& pl, const AtParams& p, int b, int h, int qi) {
  AtUnit u;
  const int tu = 2 * p.TQ;
  u.b = b;
  u.h = h;
  u.tok0 = qi * tu;
  u.ntok = pl.n[b] - u.tok0 < tu ? pl.n[b] - u.tok0 : tu;
  u.pos0 = pl.len[b] - pl.n[b] + u.tok0;
  const int end = u.pos0 + u.ntok;
  u.kv_end = end < 0 ? 0 : end;
  u.tiles = u.kv_end == 0 ? 1 : (u.kv_end + 127) / 128;
  return u;
}

// unit number u of the sequences with several: by groups of heads whose K and V fit in
// L2, then from the chunk's last tokens (the longest) to its first
__device__ __forceinline__ AtUnit at_multi_unit(const AtPlan& pl, const AtParams& p, int u) {
  int lo = 0, hi = p.c.B;  // mpre[lo] <= u < mpre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl.mpre[mid] <= u) lo = mid;
    else hi = mid;
  }
  const int Hkv = p.c.Hkv, local = u - pl.mpre[lo], nu = (pl.mpre[hi] - pl.mpre[lo]) / Hkv;
  int64_t hg = kAtL2Bytes / ((int64_t)(pl.len[lo] > 0 ? pl.len[lo] : 1) * 4 * kDim);
  hg = hg < 1 ? 1 : (hg > Hkv ? Hkv : hg);
  const int per = nu * (int)hg, gi = local / per, rem = local - gi * per;
  const int hc = Hkv - gi * (int)hg < (int)hg ? Hkv - gi * (int)hg : (int)hg;
  const int q = rem / hc;
  return at_unit(pl, p, lo, gi * (int)hg + (rem - q * hc), nu - 1 - q);
}

__device__ __forceinline__ bool at_next(const AtPlan& pl, const AtParams& p, AtWalk& w, AtSegment& s) {
  const int n = gridDim.x, c = blockIdx.x;
  if (w.wave < pl.waves) {
    s.u = at_multi_unit(pl, p, w.wave * n + ((w.wave & 1) ? n - 1 - c : c));
    ++w.wave;
    s.t0 = 0;
    s.t1 = s.u.tiles;
    s.part = false;
    return true;
  }
  if (w.x >= w.x1) return false;
  long long f0, f1;
  if (w.x < pl.Wl) {
    int lo = 0, hi = pl.left;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pl.lpre[mid] <= w.x) lo = mid;
      else hi = mid;
    }
    s.u = at_multi_unit(pl, p, pl.waves * n + lo);
    f0 = pl.lpre[lo];
    f1 = pl.lpre[lo + 1];
  } else {
    const long long y = w.x - pl.Wl;
    int lo = 0, hi = p.c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pl.spre[mid] <= y) lo = mid;
      else hi = mid;
    }
    const int tiles = (int)((pl.spre[hi] - pl.spre[lo]) / p.c.Hkv);
    const int h = (int)((y - pl.spre[lo]) / tiles);
    s.u = at_unit(pl, p, lo, h, 0);
    f0 = pl.Wl + pl.spre[lo] + (long long)h * tiles;
    f1 = f0 + tiles;
  }
  s.t0 = (int)(w.x - f0);
  const long long e = w.x1 < f1 ? w.x1 : f1;
  s.t1 = (int)(e - f0);
  w.x = e;
  s.part = s.t0 != 0 || e != f1;
  s.slot = 2 * c + (s.t0 == 0 ? 1 : 0);
  if (s.part) {  // the blocks whose shares hold the unit's first and last tile
    s.ca = (int)(((f0 + 1) * pl.shares - 1) / pl.W);
    s.cb = (int)((f1 * pl.shares - 1) / pl.W);
  }
  return true;
}

__device__ __forceinline__ void at_make_plan(AtPlan& pl, const AtParams& p, int tid) {
  const int B = p.c.B, tu = 2 * p.TQ;
  bool bad_cu = false, bad_len = false;
  for (int b = tid; b < B; b += kAtThreads) {
    int first, n;
    ragged_rows(p.c.cu_q, b, p.c.T, first, n, bad_cu);
    pl.first[b] = first;
    pl.n[b] = n;
    pl.len[b] = (int)clamp_len(p.c.seq_lens[b], p.c.geo.Nmax, bad_len);
  }
  if (bad_cu) atomicOr(p.c.err, kErrOffsets);
  if (bad_len) atomicOr(p.c.err, kErrSeqLen);
  __syncthreads();
  if (tid < 32) {
    int mu = 0;
    long long st = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + tid;
      int m = 0;
      long long s = 0;
      if (b < B && pl.n[b] > 0) {
        const int nu = (pl.n[b] + tu - 1) / tu;
        if (nu > 1) m = nu * p.c.Hkv;
        else s = (long long)p.c.Hkv * (pl.len[b] == 0 ? 1 : (pl.len[b] + 127) / 128);
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int mm = __shfl_up_sync(0xffffffffu, m, d);
        const long long ss = __shfl_up_sync(0xffffffffu, s, d);
        if (tid >= d) {
          m += mm;
          s += ss;
        }
      }
      if (b < B) {
        pl.mpre[b + 1] = mu + m;
        pl.spre[b + 1] = st + s;
      }
      mu += __shfl_sync(0xffffffffu, m, 31);
      st += __shfl_sync(0xffffffffu, s, 31);
    }
    if (tid == 0) {
      pl.mpre[0] = 0;
      pl.spre[0] = 0;
      pl.waves = mu / (int)gridDim.x;
      pl.left = mu - pl.waves * (int)gridDim.x;
    }
  }
  __syncthreads();
  if (tid < pl.left) pl.lpre[tid + 1] = at_multi_unit(pl, p, pl.waves * (int)gridDim.x + tid).tiles;
  __syncthreads();
  if (tid < 32) {
    long long sum = 0;
    for (int i0 = 1; i0 <= pl.left; i0 += 32) {
      long long v = i0 + tid <= pl.left ? pl.lpre[i0 + tid] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, d);
        if (tid >= d) v += u;
      }
      v += sum;
      if (i0 + tid <= pl.left) pl.lpre[i0 + tid] = v;
      sum = __shfl_sync(0xffffffffu, v, 31);
    }
    if (tid == 0) {
      pl.lpre[0] = 0;
      pl.Wl = sum;
      pl.W = sum + pl.spre[B];
      pl.shares = pl.W < (long long)gridDim.x ? (int)pl.W : (int)gridDim.x;  // no share is empty
    }
  }
  __syncthreads();
}

__device__ __forceinline__ AtWalk at_start(const AtPlan& pl) {
  AtWalk w;
  const int c = blockIdx.x;
  w.x = c < pl.shares ? pl.W * c / pl.shares : 0;
  w.x1 = c < pl.shares ? pl.W * (c + 1) / pl.shares : 0;
  return w;
}

__global__ void __launch_bounds__(kAtThreads, 1)
    chunk_attend_kernel(const AtParams p, const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ AtPlan pl;
  __shared__ __align__(8) uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], k_full[kAtStages],
      k_empty[kAtStages], v_full[kAtStages], v_empty[kAtStages], v_tail, all_done;
  __shared__ float2 duo[128];  // state of the second half of a one-tile unit
  __shared__ uint32_t tmem_slot, gave_up, last_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_tile = base, k_ring = base + 2 * kTileBytes, v_ring = k_ring + kAtStages * kTileBytes;

  if (tid == 0) {
    mbar_init(&q_full, 64);
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
    }
    mbar_init(&v_tail, 1);
    mbar_init(&all_done, 1);
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc512(&tmem_slot);
  tmem_fence_before();
  at_make_plan(pl, p, tid);  // ends with a barrier of the block
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;  // columns: S0 | S1 | O0 | O1, 128 each

  if (warp < 8) {
    // ------------------------------------------------------------ softmax and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    const int t = warp >> 2;                      // tile
    const int r = (warp & 3) * 32 + lane;         // row of the tile
    const uint32_t quad = (uint32_t)(warp & 3) << 21;  // 32 lanes, in the address's upper half
    const uint32_t S = tmem + quad + 128 * t, O = tmem + quad + 256 + 128 * t;
    const int G = p.c.G, rt = r / G, rg = r - rt * G;  // the row's token in the tile, its head in the group
    AtWalk w = at_start(pl);
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
            float s[128];
            {
              uint32_t x[4][32];
              tmem_ld32(S, x[0]);
              tmem_ld32(S + 32, x[1]);
              tmem_ld32(S + 64, x[2]);
              tmem_ld32(S + 96, x[3]);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(x[i >> 5][i & 31]);
            }
            if (j * 128 + 128 > vis_all) {
              const int seen = vis - j * 128;
#pragma unroll
              for (int i = 0; i < 128; ++i) s[i] = i < seen ? s[i] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int i = 4; i < 128; i += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], fmaxf(s[i + k], i + 4 + k < 128 ? s[i + 4 + k] : s[i + k]));
            }
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kScoreLog2;
            const bool raise = mt > m + 8.0f;  // also when m is -inf and a score is not
            if (__any_sync(0xffffffffu, raise)) {
              const float mn = raise ? mt : m;
              const float f = raise ? fast_exp2(m - mn) : 1.0f;  // 0 when m was -inf
              m = mn;
              l *= f;
              if (j > j0) {  // every product into O is done: S of this tile came after them
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                  uint32_t x[32];
                  tmem_ld32(O + c, x);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                  tmem_st32(O + c, x);
                }
              }
            }
            const float sub = m == -INFINITY ? 0.0f : m;
            float sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t x[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float a = fast_exp2(fmaf(s[64 * hf + 2 * i], kScoreLog2, -sub));
                const float b = fast_exp2(fmaf(s[64 * hf + 2 * i + 1], kScoreLog2, -sub));
                sum[i & 1] += a;
                sum[2 + (i & 1)] += b;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x[i]) : "f"(b), "f"(a));
              }
              tmem_st32(S + 32 * hf, x);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
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
          const int64_t row = (int64_t)(pl.first[sg.u.b] + sg.u.tok0 + tok) * p.c.Hq + sg.u.h * G + rg;
          float* st = p.part + ((int64_t)sg.slot * p.part_rows + (tok * G + rg)) * kAtPartRow;
          if (!sg.part) {
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;  // a row that sees nothing: O is 0 as well
            fa *= inv;
            fb *= inv;
          }
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t x[32];
            tmem_ld32(O + c, x);
            tmem_wait_ld();
            if (merge) {
              uint32_t y[32];
              tmem_ld32(O + 128 + c, y);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                x[i] = __float_as_uint(__uint_as_float(x[i]) * fa + __uint_as_float(y[i]) * fb);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * fa);
            }
            if (!live) continue;
            if (!sg.part) {
              uint32_t y[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                    : "=r"(y[i])
                    : "f"(__uint_as_float(x[2 * i + 1])), "f"(__uint_as_float(x[2 * i])));
              uint4* o = reinterpret_cast<uint4*>(p.c.out + row * kDim + c);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<uint4*>(st + 4 + c)[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
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
#pragma unroll 2
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
            const int64_t row = (int64_t)(pl.first[sg.u.b] + sg.u.tok0 + tk) * p.c.Hq + sg.u.h * G + (pr - tk * G);
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
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp < 12) {
      // ---------------------------------------------------------- copies
      const bool is_v = warp >= 10;
      const int lt = (tid - 256) & 63, lr = lt >> 4, lc = lt & 15;  // rows lr + 4 i, piece lc
      const uint32_t piece[2] = {tile_piece(lr, lc), tile_piece(lr + 4, lc)};  // then + 1024 every 8 rows
      const uint16_t* rows_of = (is_v ? p.c.V : p.c.K) + lc * 8;
      const uint32_t ring = is_v ? v_ring : k_ring;
      uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
      AtWalk w = at_start(pl);
      AtSegment sg;
      uint32_t it = 0, nseg = 0, tails = 0;
      bool bad = false;
      while (at_next(pl, p, w, sg)) {
        if (!is_v) {  // Q: the live rows of both tiles
          mbar_wait_or_give_up(&q_empty, (nseg & 1) ^ 1, &gave_up);
          ++nseg;
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            int rows = (sg.u.ntok - t * p.TQ) * p.c.G;
            if (rows > p.TQ * p.c.G) rows = p.TQ * p.c.G;
            const uint16_t* q = p.c.q + (int64_t)(pl.first[sg.u.b] + sg.u.tok0 + t * p.TQ) * p.c.Hq * kDim +
                                (int64_t)sg.u.h * p.c.G * kDim + lc * 8;
#pragma unroll 1
            for (int r = lr; r < rows; r += 4) {
              const int tk = r / p.c.G;
              cp_async16_or_zero(q_tile + t * kTileBytes + tile_piece(r, lc),
                                 q + ((int64_t)tk * p.c.Hq + (r - tk * p.c.G)) * kDim, true);
            }
          }
          cp_async_arrive(&q_full);
        }
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
            uint64_t* bar = zeros ? &v_tail : &full[stage];
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
              mbar_wait_or_give_up(&v_tail, tails++ & 1, &gave_up);
              for (int r = (seen < 0 ? 0 : seen) + lr; r < 128; r += 4)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + tile_piece(r, lc)), "r"(0) : "memory");
              fence_async_smem();
            }
            if (lt != 0 || zeros) mbar_arrive(&full[stage]);
            continue;
          }
          const int tb = j * 128 + lr;
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {  // rows 64 hf + lr + 4 i
            uint32_t row[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int tk = tb + 64 * hf + 4 * i;
              row[i] = tk < sg.u.kv_end ? p.c.geo.row32(sg.u.b, sg.u.h, tk, bad) : 0u;
            }
            if (hf == 0) mbar_wait_or_give_up(&empty[stage], par, &gave_up);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              cp_async16_or_zero(dst + piece[i & 1] + 8192 * hf + 1024 * (i >> 1), rows_of + (int64_t)row[i] * kDim,
                                 tb + 64 * hf + 4 * i < sg.u.kv_end);
          }
          cp_async_arrive(&full[stage]);
        }
      }
      cp_async_wait<0>();
      if (bad) atomicOr(p.c.err, kErrTable);
    } else if (warp == 12) {
      // ---------------------------------------------------------- products
      if (lane == 0) {
        AtWalk w = at_start(pl);
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
        auto outputs = [&](int t, bool acc) {
          mbar_wait_or_give_up(&p_full[t], p_par[t], &gave_up);
          p_par[t] ^= 1;
          tmem_fence_after();
          mma_probs_rows(tmem + 256 + 128 * t, tmem + 128 * t, v_ring + (iv % kAtStages) * kTileBytes, acc);
        };
        while (at_next(pl, p, w, sg)) {
          const bool two = sg.u.ntok > p.TQ;
          const int n = sg.t1 - sg.t0, ahead = two ? 1 : 2;  // K tiles whose scores are under way
          mbar_wait_or_give_up(&q_full, nseg & 1, &gave_up);
          fence_async_smem();
          ++nseg;
          for (int j = 0; j < ahead && j < n; ++j) {
            k_wait();
            tmem_fence_after();
            scores(two ? 0 : j, 0);
            if (two) scores(1, 1);
            k_next();
          }
          for (int j = 0; j < n; ++j) {
            mbar_wait_or_give_up(&v_full[iv % kAtStages], (iv / kAtStages) & 1, &gave_up);
            if (!p.box) fence_async_smem();
            const bool more = j + ahead < n;
            if (two) {
              if (more) k_wait();
              for (int t = 0; t < 2; ++t) {
                outputs(t, j > 0);
                if (more) scores(t, t);
                else mma_commit(&o_full[t]);
              }
              mma_commit(&v_empty[iv++ % kAtStages]);
              if (more) k_next();
            } else {
              const int t = j & 1;
              outputs(t, j > 1);
              mma_commit(&v_empty[iv++ % kAtStages]);
              if (more) {
                k_wait();
                scores(t, 0);
                k_next();
              } else {
                mma_commit(&o_full[t]);
              }
            }
          }
          mma_commit(&q_empty);
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
