// The attention weight each cached token received from a chunk of query rows, on the
// tensor cores: mass[t] += sum over rows of exp(q.k_t / sqrt(128) - lse[row]).
//
// A unit is 256 cached tokens of one (sequence, kv head): two tiles of 128 tokens, whose
// K rows stay in shared memory while the chunk's rows pass, 128 at a time (TQ tokens'
// heads of the group; for a short chunk from L2).  S^T = K Q^T (fp32, tensor memory) has
// a token per row, so that a thread sums its own token's weights over the columns: no
// exchange between threads, and the sums come in a fixed order.  Each token's total gets
// one addition, by one thread.  The exponentials are ex2.approx, 2 ulp of fp32: the totals
// are off by 1.8e-7 of their size, those of 32-bit exponentials summed in torch by 8e-8.
//
// A chunk of at most two Q tiles stays in shared memory over all units of its head that a
// block does one after the other (its units are then neighbours); longer chunks stream
// through the same two buffers, and a block's units are spread over the tokens, as the
// first ones are seen by more rows.
//
// Roles: warps 0-7 and 8-15 one token per thread of even and of odd units, which are at
// work at the same time (one unit's waits and ends lie in the other one's exponentials);
// warps 16-17 copy K and Q tiles (and each column's -lse log2 e); one thread of warp 18
// issues the products of even units, one of warp 19 those of odd ones.
//
// Bound by the exponentials (16 per cycle and multiprocessor) and the latency around
// them; for shorter chunks by reading K.  Measured: 64 rows of 32 heads (8 kv heads) over
// 16K-32K tokens, batch 8, 144 us (the exponentials alone 75 us, the bytes 68 us).
#pragma once

#include "chunk_attend.cuh"

namespace adamas {

constexpr int kWtThreads = 640;
constexpr int kWtStages = 2;  // of K (two tiles each) and of Q
constexpr size_t kWtSmem = (2 * kWtStages + kWtStages) * kTileBytes + 1024;

struct WtParams {
  ChunkParams c;
  int TQ, box;
};

// What a block's time goes to when the chunk's rows stay, in places of about 400 cycles: a
// unit takes kWtCostUnit and one for every 32 columns, but not less than reading its K; the
// change to another head, at which everything on its way ends first, kWtCostHead.
// (Measured a block: 2300 + 450 per 32 columns a unit, 7200 a change.  With a place for K
// and one per Q tile the slowest block took 14% longer than the mean one: 158 us where this
// takes 144, at the sizes above.)
constexpr int kWtCostRead = 8;
constexpr int kWtCostUnit = 6;
constexpr int kWtCostHead = 18;

struct WtUnit {
  int b, h, T0;      // sequence, kv head, first token
  int first, n, len; // the sequence's rows and length
  int q0, q1;        // Q tiles [q0, q1) see some of the tokens
};

// Unit number u of the launch: tab holds the units before each sequence.
__device__ __forceinline__ WtUnit wt_unit(const WtParams& p, const int* tab, int u) {
  int lo = 0, hi = p.c.B;  // tab[lo] <= u < tab[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab[mid] <= u) lo = mid;
    else hi = mid;
  }
  WtUnit w = {};
  bool bad = false;
  w.b = lo;
  ragged_rows(p.c.cu_q, lo, p.c.T, w.first, w.n, bad);
  w.len = (int)clamp_len(p.c.seq_lens[lo], p.c.geo.Nmax, bad);
  const int groups = (w.len + 255) / 256, local = u - tab[lo];
  w.h = local / groups;
  w.T0 = (local - w.h * groups) * 256;
  // row i sits at slot len - n + i and sees the slots up to it
  const int i0 = w.T0 - (w.len - w.n);
  w.q0 = i0 <= 0 ? 0 : i0 / p.TQ;
  w.q1 = (w.n + p.TQ - 1) / p.TQ;
  return w;
}

// What the copying warps tell the others with each K stage.
struct WtJob {
  int bh, T0, n, len, q0, q1;
  int q_lo;                      // first Q tile that is loaded
  bool resident, load, release;  // Q stays over units; is new; makes room after this one
  bool end;                      // no unit: the block is done
};

// The units of a block, and what becomes of the Q buffers at each (followed by the copying
// warps).
struct WtWalk {
  int u, last, step;   // unit numbers left: u, u + step, ... <= last
  int key;             // head whose Q tiles are resident (-1: none)
  uint32_t fills[2];   // of each buffer
  WtUnit w = {};

  bool resident, load, release;
  int q_lo;            // first tile that is loaded

  __device__ __forceinline__ WtWalk(const WtParams& p, const int* tab, const long long* cost, int units, bool near) {
    const int n = gridDim.x, c = blockIdx.x;
    u = near ? first_unit(p, tab, cost, cost[p.c.B] * c / n) : c;
    last = (near ? first_unit(p, tab, cost, cost[p.c.B] * (c + 1) / n) : units) - 1;
    step = near ? 1 : n;
    key = -1;
    fills[0] = fills[1] = 0;
    if (u <= last) w = wt_unit(p, tab, u);
  }
  // The first unit that begins at or behind place x when the places of sequence b are
  // [cost[b], cost[b + 1]): for each head the change to it and its units.
  static __device__ __forceinline__ int first_unit(const WtParams& p, const int* tab, const long long* cost, long long x) {
    int lo = 0, hi = p.c.B;  // cost[lo] <= x < cost[hi], or x is the end
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cost[mid] <= x) lo = mid;
      else hi = mid;
    }
    const int groups = (tab[lo + 1] - tab[lo]) / p.c.Hkv;
    if (groups == 0) return tab[lo];
    const long long head = (cost[lo + 1] - cost[lo]) / p.c.Hkv, each = (head - kWtCostHead) / groups;
    const long long h = (x - cost[lo]) / head, in = x - cost[lo] - h * head - kWtCostHead;
    return tab[lo] + (int)h * groups + (in <= 0 ? 0 : (int)((in + each - 1) / each));
  }
  __device__ __forceinline__ bool stays(const WtUnit& x) const { return x.q1 <= 2; }
  // prepares the unit at hand; false: none left
  __device__ __forceinline__ bool begin(const WtParams& p, const int* tab, WtUnit& next) {
    if (u > last) return false;
    const int head = w.b * p.c.Hkv + w.h;
    resident = stays(w);
    load = !resident || head != key;
    key = resident ? head : -1;
    q_lo = resident ? 0 : w.q0;
    release = true;
    if (u + step <= last) {
      next = wt_unit(p, tab, u + step);
      release = !(resident && stays(next) && next.b == w.b && next.h == w.h);
    }
    return true;
  }
  __device__ __forceinline__ void end(const WtUnit& next) {
    u += step;
    w = next;
  }
};

__global__ void __launch_bounds__(kWtThreads, 1)
    chunk_weights_kernel(const WtParams p, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ int tab[kMaxBatch + 1];         // units before each sequence
  __shared__ long long cost[kMaxBatch + 1];  // and what they cost, in places
  __shared__ __align__(16) float neg_lse[kWtStages][128];
  __shared__ __align__(8) uint64_t k_full[kWtStages], k_empty[kWtStages], q_full[kWtStages], q_empty[kWtStages],
      s_full[2][2], s_empty[2][2], all_done;
  __shared__ WtJob jobs[kWtStages];
  __shared__ uint32_t tmem_slot, gave_up;
  __shared__ int longest;  // chunk of the batch
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t k_ring = base, q_ring = base + 2 * kWtStages * kTileBytes;

  if (tid == 0) {
    for (int i = 0; i < kWtStages; ++i) {
      mbar_init(&k_full[i], 64);
      mbar_init(&k_empty[i], 2 + 16);  // the products and the readers of the job
      mbar_init(&q_full[i], 64);
      mbar_init(&q_empty[i], 2 + 16);  // the products and the readers of neg_lse
    }
    for (int t = 0; t < 2; ++t)
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[t][i], 1);
        mbar_init(&s_empty[t][i], 4);
      }
    mbar_init(&all_done, 2);
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 18) tmem_alloc512(&tmem_slot);
  if (warp == 0) {  // units before each sequence
    int all = 0, most = 0;
    long long places = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
      int s = 0;
      long long z = 0;
      if (b0 + lane < p.c.B) {
        bool bad_cu = false, bad_len = false;
        int first, n;
        ragged_rows(p.c.cu_q, b0 + lane, p.c.T, first, n, bad_cu);
        const int len = (int)clamp_len(p.c.seq_lens[b0 + lane], p.c.geo.Nmax, bad_len);
        if (bad_cu) atomicOr(p.c.err, kErrOffsets);
        if (bad_len) atomicOr(p.c.err, kErrSeqLen);
        if (n > 0) s = (len + 255) / 256 * p.c.Hkv;
        if (s > 0)
          z = (long long)p.c.Hkv * kWtCostHead +
              (long long)s * max(kWtCostRead, kWtCostUnit + (min(n, 2 * p.TQ) * p.c.G + 31) / 32);
        most = n > most ? n : most;
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, d);
        const long long y = __shfl_up_sync(0xffffffffu, z, d);
        if (lane >= d) {
          s += u;
          z += y;
        }
      }
      s += all;
      z += places;
      if (b0 + lane < p.c.B) {
        tab[b0 + lane + 1] = s;
        cost[b0 + lane + 1] = z;
      }
      all = __shfl_sync(0xffffffffu, s, 31);
      places = __shfl_sync(0xffffffffu, z, 31);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      tab[0] = 0;
      cost[0] = 0;
      longest = most;
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;  // columns: tile 0's two S, tile 1's two S, 128 each
  const int units = tab[p.c.B];

  if (warp < 16) {
    // ------------------------------------------------------------ sums of weights
    const int t = (warp >> 2) & 1, buf = warp >> 3, r = (warp & 3) * 32 + lane, G = p.c.G;
    const uint32_t from = tmem + ((uint32_t)(warp & 3) << 21) + 256 * t + 128 * buf;
    uint32_t is = 0, fills[2] = {0, 0};  // S taken, fills of the Q buffers
    for (uint32_t ik = 0;; ++ik) {
      const uint32_t ks = ik % kWtStages;
      mbar_wait_or_give_up(&k_full[ks], (ik / kWtStages) & 1, &gave_up);
      const WtJob w = jobs[ks];
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_empty[ks]);
      if (w.end || *(volatile uint32_t*)&gave_up) break;
      const bool mine = ks == (uint32_t)buf;
      const int slot = w.T0 + 128 * t + r;
      const bool tile = mine && w.T0 + 128 * t < w.len;
      float* out = p.c.mass + (int64_t)w.bh * p.c.geo.Nmax + slot;
      uint64_t sum[4] = {0, 0, 0, 0};
      if (w.load && w.resident) {
        ++fills[0];
        if (w.q1 > 1) ++fills[1];
      }
      for (int q = w.q0; q < w.q1; ++q) {
        const uint32_t stage = (q - w.q_lo) & 1;
        if (!w.resident) ++fills[stage];
        if (mine || !w.resident)  // neg_lse is there
          mbar_wait_or_give_up(&q_full[stage], (fills[stage] - 1) & 1, &gave_up);
        if (tile) {
          mbar_wait_or_give_up(&s_full[t][buf], is++ & 1, &gave_up);
          tmem_fence_after();
          // the columns that see the slot: those of the tokens at or behind it
          const int tok0 = q * p.TQ, toks = w.n - tok0 < p.TQ ? w.n - tok0 : p.TQ;
          const int c1 = toks * G;
          int c0 = (slot - (w.len - w.n) - tok0) * G;
          c0 = slot >= w.len ? 128 : (c0 < 0 ? 0 : c0);
          const bool some = __any_sync(0xffffffffu, c0 > 0);
          const uint64_t scale2 = f2_pack(kScoreLog2, kScoreLog2);
          const uint32_t nl = smem_addr(&neg_lse[stage][0]);
          // 32 columns at a time, the next ones on their way meanwhile
          uint32_t xa[32], xb[32];
          auto add = [&](uint32_t (&x)[32], int i0) {
#pragma unroll
            for (int hf = 0; hf < 32; hf += 16) {
              if (i0 + hf >= c1) break;
              if (some || i0 + hf + 16 > c1) {  // columns that do not see the slot: a score of -inf
#pragma unroll
                for (int i = hf; i < hf + 16; ++i) x[i] = i0 + i >= c0 && i0 + i < c1 ? x[i] : 0xFF800000u;
              }
              uint4 z[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) z[i] = lds128(nl + 4 * (i0 + hf) + 16 * i);
              float e[16];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int n = hf + 4 * i;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(x[n]), __uint_as_float(x[n + 1])), scale2,
                                 f2_pack(__uint_as_float(z[i].x), __uint_as_float(z[i].y))),
                          e[4 * i], e[4 * i + 1]);
                f2_unpack(f2_fma(f2_pack(__uint_as_float(x[n + 2]), __uint_as_float(x[n + 3])), scale2,
                                 f2_pack(__uint_as_float(z[i].z), __uint_as_float(z[i].w))),
                          e[4 * i + 2], e[4 * i + 3]);
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) e[i] = fast_exp2(e[i]);
#pragma unroll
              for (int i = 0; i < 8; ++i) sum[i & 3] = f2_add(sum[i & 3], f2_pack(e[2 * i], e[2 * i + 1]));
            }
          };
          tmem_ld32(from, xa);
          tmem_wait_ld(xa);
          tmem_ld32(from + 32, xb);
          add(xa, 0);
          tmem_wait_ld(xb);
          tmem_ld32(from + 64, xa);
          add(xb, 32);
          tmem_wait_ld(xa);
          tmem_ld32(from + 96, xb);
          add(xa, 64);
          tmem_wait_ld(xb);
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[t][buf]);
          add(xb, 96);
        }
        if (!w.resident) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_empty[stage]);
        }
      }
      if (mine && slot < w.len) {
        float a, b;
        f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), a, b);
        atomicAdd(out, a + b);  // the one addition to this token: nothing to wait for
      }
      if (w.resident && w.release) {  // not before the buffers were filled: this may be the unit they are for
        mbar_wait_or_give_up(&q_full[0], (fills[0] - 1) & 1, &gave_up);
        if (w.q1 > 1) mbar_wait_or_give_up(&q_full[1], (fills[1] - 1) & 1, &gave_up);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&q_empty[0]);
          if (w.q1 > 1) mbar_arrive(&q_empty[1]);
        }
      }
    }
  } else if (warp < 18) {
    // ------------------------------------------------------------ copies
    const int lt = tid - 512, lr = lt >> 4, lc = lt & 15;
    WtWalk k = WtWalk(p, tab, cost, units, longest <= 2 * p.TQ);
    WtUnit next;
    uint32_t ik = 0;
    bool bad = false;
    auto publish = [&](uint32_t stage, bool end) {  // by the thread that arrives first
      const WtUnit& w = k.w;
      jobs[stage] = WtJob{w.b * p.c.Hkv + w.h, w.T0, w.n, w.len, w.q0, w.q1, k.q_lo, k.resident, k.load, k.release, end};
    };
    for (; k.begin(p, tab, next); ++ik) {
      const WtUnit& w = k.w;
      const uint32_t stage = ik % kWtStages, dst = k_ring + 2 * stage * kTileBytes;
      const int rows = w.len - w.T0 < 256 ? w.len - w.T0 : 256;
      if (p.box) {
        const int pieces = (rows + p.box - 1) / p.box;  // at most 32
        uint32_t row = 0;
        if (lt < pieces) row = p.c.geo.row32(w.b, w.h, w.T0 + lt * p.box, bad);
        mbar_wait_or_give_up(&k_empty[stage], ((ik / kWtStages) & 1) ^ 1, &gave_up);
        if (lt == 0) {
          publish(stage, false);
          mbar_arrive_expect_tx(&k_full[stage], (uint32_t)(pieces * p.box * 2 * kDim));
        }
        if (lt < 32) {
          __syncwarp();
          if (lt < pieces) {
            const int r = lt * p.box;
            const uint32_t at = dst + (r >> 7) * kTileBytes + (r & 127) * 128;
            tma_load_2d(at, &k_map, 0, (int)row, &k_full[stage]);
            tma_load_2d(at + kTileHalf, &k_map, 64, (int)row, &k_full[stage]);
          }
        }
        if (lt != 0) mbar_arrive(&k_full[stage]);
      } else {
        mbar_wait_or_give_up(&k_empty[stage], ((ik / kWtStages) & 1) ^ 1, &gave_up);
        if (lt == 0) publish(stage, false);
#pragma unroll 4
        for (int r = lr; r < rows; r += 4) {
          const uint32_t row = p.c.geo.row32(w.b, w.h, w.T0 + r, bad);
          cp_async16_or_zero(dst + (r >> 7) * kTileBytes + tile_piece(r & 127, lc), p.c.K + (int64_t)row * kDim + lc * 8, true);
        }
        cp_async_arrive(&k_full[stage]);
      }
      for (int q = k.q_lo; q < w.q1 && k.load; ++q) {
        const uint32_t qs = (q - k.q_lo) & 1;
        const int tok0 = q * p.TQ, cols = (w.n - tok0 < p.TQ ? w.n - tok0 : p.TQ) * p.c.G;
        float z[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // a column without a row, or whose row saw nothing, gives 2^-inf
          const int c = lt + 64 * j, tk = c / p.c.G;
          z[j] = -INFINITY;
          if (c < cols) {
            const float v = p.c.lse[(int64_t)(w.first + tok0 + tk) * p.c.Hq + w.h * p.c.G + (c - tk * p.c.G)];
            if (v != -INFINITY) z[j] = -v * 1.4426950408889634f;
          }
        }
        mbar_wait_or_give_up(&q_empty[qs], (k.fills[qs]++ & 1) ^ 1, &gave_up);
        neg_lse[qs][lt] = z[0];
        neg_lse[qs][lt + 64] = z[1];
        if (lt == 0) {
          mbar_arrive_expect_tx(&q_full[qs], (uint32_t)(p.TQ * p.c.G * 2 * kDim));
          tma_load_3d(q_ring + qs * kTileBytes, &q_map, 0, w.h * p.c.G, w.first + tok0, &q_full[qs]);
          tma_load_3d(q_ring + qs * kTileBytes + kTileHalf, &q_map, 64, w.h * p.c.G, w.first + tok0, &q_full[qs]);
        } else {
          mbar_arrive(&q_full[qs]);
        }
      }
      k.end(next);
    }
    mbar_wait_or_give_up(&k_empty[ik % kWtStages], ((ik / kWtStages) & 1) ^ 1, &gave_up);
    if (lt == 0) publish(ik % kWtStages, true);
    mbar_arrive(&k_full[ik % kWtStages]);
    cp_async_wait<0>();
    // the copies land before the block goes, also when somebody gave up waiting for them
    for (uint32_t i = 0; i < kWtStages; ++i) {  // the last phase of each barrier
      if (ik >= i) mbar_wait_timed(&k_full[(ik - i) % kWtStages], ((ik - i) / kWtStages) & 1, 1000000000ull);
      if (k.fills[i] > 0) mbar_wait_timed(&q_full[i], (k.fills[i] - 1) & 1, 1000000000ull);
    }
    if (bad) atomicOr(p.c.err, kErrTable);
  } else if (lane == 0) {
    // ------------------------------------------------------------ products
    const uint32_t buf = warp - 18;
    uint32_t made[2] = {0, 0}, fills[2] = {0, 0};  // S of each tile, fills of the Q buffers
    for (uint32_t ik = 0;; ++ik) {
      const uint32_t stage = ik % kWtStages, kt = k_ring + 2 * stage * kTileBytes;
      mbar_wait_or_give_up(&k_full[stage], (ik / kWtStages) & 1, &gave_up);
      const WtJob w = jobs[stage];
      if (w.end || *(volatile uint32_t*)&gave_up) break;
      const bool mine = stage == buf;
      if (!mine) mbar_arrive(&k_empty[stage]);
      if (!p.box) fence_async_smem();
      const int nt = w.T0 + 128 < w.len ? 2 : 1;
      if (w.load && w.resident) {
        ++fills[0];
        if (w.q1 > 1) ++fills[1];
      }
      for (int q = w.q0; q < w.q1 && (mine || !w.resident); ++q) {
        const uint32_t qs = (q - w.q_lo) & 1;
        if (!w.resident) ++fills[qs];
        mbar_wait_or_give_up(&q_full[qs], (fills[qs] - 1) & 1, &gave_up);
        if (!mine) {
          mbar_arrive(&q_empty[qs]);
          continue;
        }
        for (int t = 0; t < nt; ++t) {
          mbar_wait_or_give_up(&s_empty[t][buf], (made[t]++ & 1) ^ 1, &gave_up);
          tmem_fence_after();
          mma_rows_rows(tmem + 256 * t + 128 * buf, kt + t * kTileBytes, q_ring + qs * kTileBytes);
          mma_commit(&s_full[t][buf]);
        }
        if (!w.resident) mma_commit(&q_empty[qs]);
      }
      if (mine) mma_commit(&k_empty[stage]);
      if (w.resident && w.release) {  // (what the thread issued for units before is done then, too)
        mbar_wait_or_give_up(&q_full[0], (fills[0] - 1) & 1, &gave_up);
        if (w.q1 > 1) mbar_wait_or_give_up(&q_full[1], (fills[1] - 1) & 1, &gave_up);
        mma_commit(&q_empty[0]);
        if (w.q1 > 1) mma_commit(&q_empty[1]);
      }
    }
    mma_commit(&all_done);
    mbar_wait_or_give_up(&all_done, 0, &gave_up);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 18) tmem_free512(tmem);
  if (tid == 0 && gave_up) atomicOr(p.c.err, kErrTimeout);
}

}  // namespace adamas
