// The attention weight each cached token received from a chunk of query rows, on the
// tensor cores: mass[t] += sum over rows of exp(q.k_t / sqrt(128) - lse[row]).
//
// A unit is 256 cached tokens of one (sequence, kv head): two tiles of 128 tokens, whose
// K rows stay in shared memory while the chunk's rows pass, 128 at a time (TQ tokens'
// heads of the group; for a short chunk from L2).  S^T = K Q^T (fp32, tensor memory) has
// a token per row, so that a thread sums its own token's weights over the columns: no
// exchange between threads, and the sums come in a fixed order.  Each token's total is
// read and written once, by one thread.
//
// Roles: warps 0-3 and 4-7 one token per thread of tile 0 and 1; warps 8-9 copy K and Q
// tiles (and each column's -lse log2 e); one thread of warp 10 issues the products, two
// S per tile, so that one is summed while the other is made.
//
// Bound by the exponentials (16 per cycle and multiprocessor) or, for short chunks, by
// reading K.
#pragma once

#include "chunk_attend.cuh"

namespace adamas {

constexpr int kWtThreads = 352;
constexpr int kWtStages = 2;  // of K (two tiles each) and of Q
constexpr size_t kWtSmem = (2 * kWtStages + kWtStages) * kTileBytes + 1024;

struct WtParams {
  ChunkParams c;
  int TQ, box;
};

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
  WtUnit w;
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

__global__ void __launch_bounds__(kWtThreads, 1)
    chunk_weights_kernel(const WtParams p, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ int tab[kMaxBatch + 1];
  __shared__ __align__(16) float neg_lse[kWtStages][128];
  __shared__ __align__(8) uint64_t k_full[kWtStages], k_empty[kWtStages], q_full[kWtStages], q_empty[kWtStages],
      s_full[2][2], s_empty[2][2], all_done;
  __shared__ uint32_t tmem_slot, gave_up;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t k_ring = base, q_ring = base + 2 * kWtStages * kTileBytes;

  if (tid == 0) {
    for (int i = 0; i < kWtStages; ++i) {
      mbar_init(&k_full[i], 64);
      mbar_init(&k_empty[i], 1);
      mbar_init(&q_full[i], 64);
      mbar_init(&q_empty[i], 1 + 8);  // the products and the readers of neg_lse
    }
    for (int t = 0; t < 2; ++t)
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[t][i], 1);
        mbar_init(&s_empty[t][i], 4);
      }
    mbar_init(&all_done, 1);
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 10) tmem_alloc512(&tmem_slot);
  if (warp == 0) {  // units before each sequence
    int all = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
      int s = 0;
      if (b0 + lane < p.c.B) {
        bool bad_cu = false, bad_len = false;
        int first, n;
        ragged_rows(p.c.cu_q, b0 + lane, p.c.T, first, n, bad_cu);
        const int len = (int)clamp_len(p.c.seq_lens[b0 + lane], p.c.geo.Nmax, bad_len);
        if (bad_cu) atomicOr(p.c.err, kErrOffsets);
        if (bad_len) atomicOr(p.c.err, kErrSeqLen);
        if (n > 0) s = (len + 255) / 256 * p.c.Hkv;
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += u;
      }
      s += all;
      if (b0 + lane < p.c.B) tab[b0 + lane + 1] = s;
      all = __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) tab[0] = 0;
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;  // columns: tile 0's two S, tile 1's two S, 128 each
  const int units = tab[p.c.B];

  if (warp < 8) {
    // ------------------------------------------------------------ sums of weights
    const int t = warp >> 2, r = (warp & 3) * 32 + lane, G = p.c.G;
    const uint32_t S = tmem + ((uint32_t)(warp & 3) << 21) + 256 * t;
    uint32_t is = 0, iq = 0;  // S of this tile, Q tiles
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const WtUnit w = wt_unit(p, tab, u);
      const int slot = w.T0 + 128 * t + r;
      const bool tile = w.T0 + 128 * t < w.len;
      float* out = p.c.mass + ((int64_t)w.b * p.c.Hkv + w.h) * p.c.geo.Nmax + slot;
      float before = 0.0f;
      if (slot < w.len) before = *out;
      uint64_t sum[2] = {0, 0};
      for (int q = w.q0; q < w.q1; ++q, ++iq) {
        const uint32_t stage = iq % kWtStages;
        mbar_wait_or_give_up(&q_full[stage], (iq / kWtStages) & 1, &gave_up);  // neg_lse is there
        if (tile) {
          mbar_wait_or_give_up(&s_full[t][is & 1], (is >> 1) & 1, &gave_up);
          tmem_fence_after();
          // the columns that see the slot: those of the tokens at or behind it
          const int tok0 = q * p.TQ, toks = w.n - tok0 < p.TQ ? w.n - tok0 : p.TQ;
          const int c1 = toks * G;
          int c0 = (slot - (w.len - w.n) - tok0) * G;
          c0 = slot >= w.len ? 128 : (c0 < 0 ? 0 : c0);
          const bool edge = __any_sync(0xffffffffu, c0 > 0) || c1 < 128;
          const uint32_t from = S + 128 * (is & 1);
          uint32_t x[4][32];
          tmem_ld32(from, x[0]);
          tmem_ld32(from + 32, x[1]);
          tmem_ld32(from + 64, x[2]);
          tmem_ld32(from + 96, x[3]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(x[c]);
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[t][is & 1]);
          const uint64_t scale2 = f2_pack(kScoreLog2, kScoreLog2);
          const uint32_t nl = smem_addr(&neg_lse[stage][0]);
#pragma unroll
          for (int i = 0; i < 128; i += 4) {
            const uint4 z = lds128(nl + 4 * i);
            const uint64_t e0 = f2_fma(f2_pack(__uint_as_float(x[i >> 5][i & 31]), __uint_as_float(x[i >> 5][(i & 31) + 1])),
                                       scale2, f2_pack(__uint_as_float(z.x), __uint_as_float(z.y)));
            const uint64_t e1 = f2_fma(f2_pack(__uint_as_float(x[i >> 5][(i & 31) + 2]), __uint_as_float(x[i >> 5][(i & 31) + 3])),
                                       scale2, f2_pack(__uint_as_float(z.z), __uint_as_float(z.w)));
            float a, b, c, d;
            f2_unpack(e0, a, b);
            f2_unpack(e1, c, d);
            a = fast_exp2(a);
            b = fast_exp2(b);
            c = fast_exp2(c);
            d = fast_exp2(d);
            if (edge) {
              a = i >= c0 && i < c1 ? a : 0.0f;
              b = i + 1 >= c0 && i + 1 < c1 ? b : 0.0f;
              c = i + 2 >= c0 && i + 2 < c1 ? c : 0.0f;
              d = i + 3 >= c0 && i + 3 < c1 ? d : 0.0f;
            }
            sum[0] = f2_add(sum[0], f2_pack(a, b));
            sum[1] = f2_add(sum[1], f2_pack(c, d));
          }
          ++is;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[stage]);
      }
      if (slot < w.len) {
        float a, b;
        f2_unpack(f2_add(sum[0], sum[1]), a, b);
        *out = before + (a + b);
      }
    }
  } else if (warp < 10) {
    // ------------------------------------------------------------ copies
    const int lt = tid - 256, lr = lt >> 4, lc = lt & 15;
    uint32_t ik = 0, iq = 0;
    bool bad = false;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++ik) {
      const WtUnit w = wt_unit(p, tab, u);
      const uint32_t stage = ik % kWtStages, dst = k_ring + 2 * stage * kTileBytes;
      const int rows = w.len - w.T0 < 256 ? w.len - w.T0 : 256;
      if (p.box) {
        const int pieces = (rows + p.box - 1) / p.box;  // at most 32
        uint32_t row = 0;
        if (lt < pieces) row = p.c.geo.row32(w.b, w.h, w.T0 + lt * p.box, bad);
        mbar_wait_or_give_up(&k_empty[stage], ((ik / kWtStages) & 1) ^ 1, &gave_up);
        if (lt == 0) mbar_arrive_expect_tx(&k_full[stage], (uint32_t)(pieces * p.box * 2 * kDim));
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
#pragma unroll 4
        for (int r = lr; r < rows; r += 4) {
          const uint32_t row = p.c.geo.row32(w.b, w.h, w.T0 + r, bad);
          cp_async16_or_zero(dst + (r >> 7) * kTileBytes + tile_piece(r & 127, lc), p.c.K + (int64_t)row * kDim + lc * 8, true);
        }
        cp_async_arrive(&k_full[stage]);
      }
      for (int q = w.q0; q < w.q1; ++q, ++iq) {
        const uint32_t qs = iq % kWtStages;
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
        mbar_wait_or_give_up(&q_empty[qs], ((iq / kWtStages) & 1) ^ 1, &gave_up);
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
    }
    cp_async_wait<0>();
    if (bad) atomicOr(p.c.err, kErrTable);
  } else if (lane == 0) {
    // ------------------------------------------------------------ products
    uint32_t ik = 0, iq = 0, is[2] = {0, 0};
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++ik) {
      const WtUnit w = wt_unit(p, tab, u);
      const uint32_t stage = ik % kWtStages, k = k_ring + 2 * stage * kTileBytes;
      const int nt = w.T0 + 128 < w.len ? 2 : 1;
      mbar_wait_or_give_up(&k_full[stage], (ik / kWtStages) & 1, &gave_up);
      if (!p.box) fence_async_smem();
      for (int q = w.q0; q < w.q1; ++q, ++iq) {
        const uint32_t qs = iq % kWtStages;
        mbar_wait_or_give_up(&q_full[qs], (iq / kWtStages) & 1, &gave_up);
        for (int t = 0; t < nt; ++t) {
          mbar_wait_or_give_up(&s_empty[t][is[t] & 1], ((is[t] >> 1) & 1) ^ 1, &gave_up);
          tmem_fence_after();
          mma_rows_rows(tmem + 256 * t + 128 * (is[t] & 1), k + t * kTileBytes, q_ring + qs * kTileBytes);
          mma_commit(&s_full[t][is[t] & 1]);
          ++is[t];
        }
        mma_commit(&q_empty[qs]);
      }
      mma_commit(&k_empty[stage]);
    }
    mma_commit(&all_done);
    mbar_wait_or_give_up(&all_done, 0, &gave_up);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 10) tmem_free512(tmem);
  if (tid == 0 && gave_up) atomicOr(p.c.err, kErrTimeout);
}

}  // namespace adamas
