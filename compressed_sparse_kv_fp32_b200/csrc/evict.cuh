// Attention weight of the decode step's kept tokens, and the eviction of the tokens
// with the least accumulated weight.
#pragma once

#include <cooperative_groups.h>

#include "cache.cuh"
#include "chunk.cuh"
#include "umma.cuh"

namespace adamas {

struct KeptParams {
  const uint16_t *q, *K;
  const int32_t *idx, *seq_lens;
  int B, Hq, Hkv, G, budget, shared_rows;
  float* mass;
  CacheGeom geo;
  uint32_t* err;
};

// A cluster of blocks per (b, kv head), a share of every list each; sixteen lanes make a
// score (one K row, 16 bytes a lane), four of them under way at a time, and the scores
// stay in shared memory.  The blocks exchange maxima and sums; then the weights are added
// to mass list after list, a barrier of the cluster between two lists, so that the weights
// of two heads that kept the same token are added in a fixed order.  A list the query
// heads share is read once, and its tokens get the heads' weights in one addition.  The
// exponentials are ex2.approx, 2 ulp of fp32.
// Bound by latency, then by the K rows.  Measured: 32 heads of 1024 kept tokens of 128K
// 7.7 us (8.8 MB; one block a head and the scores made three times: 34 us).
constexpr int kKeptThreads = 256;
constexpr int kKeptCluster = 8;
constexpr int kKeptSmemFloats = 49152;

__global__ void __launch_bounds__(kKeptThreads) accumulate_kept_kernel(const KeptParams p, int cap) {
  namespace cg = cooperative_groups;
  constexpr int kHalves = kKeptThreads / 16, kAhead = 4;
  extern __shared__ float sm_score[];  // [G][cap]
  __shared__ float sq[kMaxGroup][kDim];
  __shared__ float red[kMaxGroup][kHalves];
  __shared__ float2 state[kMaxGroup];  // this block's maximum and sum of each head
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid & 15, half = tid >> 4;
  const int hk = blockIdx.x / C, b = hk / p.Hkv, kvh = hk - b * p.Hkv;
  bool badlen = false, badpage = false;
  const int len = (int)clamp_len(p.seq_lens[b], p.geo.Nmax, badlen);
  if (badlen && tid == 0) atomicOr(p.err, kErrSeqLen);
  const int lists = p.shared_rows ? 1 : p.G, heads = p.shared_rows ? p.G : 1;
  const int i0 = (int)((int64_t)rank * p.budget / C), n = (int)((int64_t)(rank + 1) * p.budget / C) - i0;
  auto list = [&](int g) { return p.idx + (p.shared_rows ? (int64_t)hk : (int64_t)b * p.Hq + kvh * p.G + g) * p.budget + i0; };
  for (int i = tid; i < p.G * kDim; i += kKeptThreads)
    sq[i / kDim][i % kDim] =
        __uint_as_float((uint32_t)p.q[((int64_t)b * p.Hq + kvh * p.G) * kDim + i] << 16) * kScoreLog2;
  __syncthreads();
  for (int g = 0; g < lists; ++g) {
    const int32_t* idx = list(g);
    float m[kMaxGroup];
#pragma unroll
    for (int a = 0; a < kMaxGroup; ++a) m[a] = -INFINITY;
    for (int s0 = half; s0 - half < n; s0 += kAhead * kHalves) {  // the same number of rounds in both halves of a warp
      int t[kAhead];
      uint4 w[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int s = s0 + j * kHalves;
        t[j] = s < n ? idx[s] : -1;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (t[j] >= len) t[j] = -1;
        w[j] = make_uint4(0, 0, 0, 0);
        if (t[j] >= 0) w[j] = reinterpret_cast<const uint4*>(p.K + p.geo.row(b, kvh, t[j], badpage) * kDim)[l];
      }
#pragma unroll
      for (int a = 0; a < kMaxGroup; ++a) {
        if (a >= heads) break;
        const float4 qa = *reinterpret_cast<const float4*>(&sq[g + a][8 * l]);
        const float4 qb = *reinterpret_cast<const float4*>(&sq[g + a][8 * l + 4]);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          float d = qa.x * bf16_lo(w[j].x) + qa.y * bf16_hi(w[j].x) + qa.z * bf16_lo(w[j].y) + qa.w * bf16_hi(w[j].y) +
                    qb.x * bf16_lo(w[j].z) + qb.y * bf16_hi(w[j].z) + qb.z * bf16_lo(w[j].w) + qb.w * bf16_hi(w[j].w);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
          if (t[j] < 0) d = -INFINITY;
          m[a] = fmaxf(m[a], d);
          const int s = s0 + j * kHalves;
          if (l == 0 && s < n) sm_score[(g + a) * cap + s] = d;
        }
      }
    }
#pragma unroll
    for (int a = 0; a < kMaxGroup; ++a)
      if (a < heads && l == 0) red[g + a][half] = m[a];
  }
  __syncthreads();
  if (warp < p.G) {  // a warp per head: the block's maximum and sum
    float m = lane < kHalves ? red[warp][lane] : -INFINITY;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = __shfl_sync(0xffffffffu, m, 0);
    float sum = 0.0f;
    if (m != -INFINITY)
      for (int s = lane; s < n; s += 32) sum += fast_exp2(sm_score[warp * cap + s] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) state[warp] = make_float2(m, sum);
  }
  cluster.sync();
  float* mass = p.mass + (int64_t)hk * p.geo.Nmax;
  for (int g = 0; g < lists; ++g) {
    float M[kMaxGroup], inv[kMaxGroup];
#pragma unroll
    for (int a = 0; a < kMaxGroup; ++a) {
      M[a] = -INFINITY;
      inv[a] = 0.0f;
      if (a < heads) {
        float L = 0.0f;
        for (int c = 0; c < C; ++c) M[a] = fmaxf(M[a], cluster.map_shared_rank(state, c)[g + a].x);
        for (int c = 0; c < C; ++c) {
          const float2 st = cluster.map_shared_rank(state, c)[g + a];
          if (st.x != -INFINITY) L += st.y * fast_exp2(st.x - M[a]);
        }
        if (L > 0.0f) inv[a] = 1.0f / L;
      }
    }
    const int32_t* idx = list(g);
    for (int s = tid; s < n; s += kKeptThreads) {
      const int t = idx[s];
      if (t < 0 || t >= len) continue;
      float w = 0.0f;
#pragma unroll
      for (int a = 0; a < kMaxGroup; ++a)
        if (a < heads) w += fast_exp2(sm_score[(g + a) * cap + s] - M[a]) * inv[a];
      atomicAdd(mass + t, w);
    }
    cluster.sync();  // before the next list's additions; at the end, before any block's shared memory goes
  }
  if (badpage) atomicOr(p.err, kErrTable);
}

// Lists too long for the scores to stay in the cluster's shared memory: one block per
// (b, kv head), the scores made anew for the maximum, the sum and the weights.
__global__ void __launch_bounds__(256) accumulate_kept_large_kernel(const KeptParams p) {
  __shared__ float sq[kDim];
  __shared__ float red[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x, b = hk / p.Hkv, kvh = hk - b * p.Hkv;
  bool badlen = false, badpage = false;
  const int64_t len = clamp_len(p.seq_lens[b], p.geo.Nmax, badlen);
  if (badlen && tid == 0) atomicOr(p.err, kErrSeqLen);
  float* mass = p.mass + (int64_t)hk * p.geo.Nmax;
  for (int g = 0; g < p.G; ++g) {
    const int h = kvh * p.G + g;
    const int32_t* idx = p.idx + (p.shared_rows ? (int64_t)hk : (int64_t)b * p.Hq + h) * p.budget;
    __syncthreads();
    if (tid < kDim) sq[tid] = __uint_as_float((uint32_t)p.q[((int64_t)b * p.Hq + h) * kDim + tid] << 16);
    __syncthreads();
    auto score = [&](int t) {
      const uint4* k = reinterpret_cast<const uint4*>(p.K + p.geo.row(b, kvh, t, badpage) * kDim);
      float a = 0.0f;
      for (int c = 0; c < 16; ++c) {
        const uint4 w = k[c];
        const float* qq = &sq[8 * c];
        a += qq[0] * bf16_lo(w.x) + qq[1] * bf16_hi(w.x) + qq[2] * bf16_lo(w.y) + qq[3] * bf16_hi(w.y) +
             qq[4] * bf16_lo(w.z) + qq[5] * bf16_hi(w.z) + qq[6] * bf16_lo(w.w) + qq[7] * bf16_hi(w.w);
      }
      return a * kScoreLog2;
    };
    float m = -INFINITY;
    for (int i = tid; i < p.budget; i += 256) {
      const int t = idx[i];
      if (t >= 0 && t < len) m = fmaxf(m, score(t));
    }
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
    __syncthreads();
    float l = 0.0f;
    for (int i = tid; i < p.budget; i += 256) {
      const int t = idx[i];
      if (t >= 0 && t < len) l += exp2f(score(t) - m);
    }
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane == 0) red[warp] = l;
    __syncthreads();
    l = 0.0f;
    for (int w = 0; w < 8; ++w) l += red[w];
    for (int i = tid; i < p.budget; i += 256) {
      const int t = idx[i];
      if (t >= 0 && t < len) atomicAdd(mass + t, exp2f(score(t) - m) / l);
    }
  }
  if (badpage) atomicOr(p.err, kErrTable);
}

struct EvictParams {
  const uint16_t *K, *V;
  const uint8_t* codes;
  const float* mass;
  const int32_t* seq_lens;
  int B, Hkv, keep, n_sink, n_recent;
  int32_t *kept, *new_lens;
  uint16_t *K_out, *V_out;
  uint8_t* codes_out;
  float* mass_out;
  int smem_keys;  // keys of a slice that the selection's launch has shared memory for
  CacheGeom geo, out;
  uint32_t* err;
};

// Order-preserving image of a mass in unsigned integers: larger is kept first.  -0 is
// 0; NaN is below everything; forced tokens are above everything.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// ---------------------------------------------------------------- which tokens stay
// A cluster of blocks per (b, kv head), a slice of the tokens each.  The keys are read
// once into shared memory (a slice that does not fit what the launch has is read again).
// The k-th largest key is found by 8-bit digits, most significant first: the blocks count
// their keys under the digits known so far, each adds up the cluster's counts, and one warp
// finds the digit; the rest of the digits need not be known once all keys under them are
// kept.  Then every warp counts what it keeps of its run of tokens, and writes the kept
// slots in ascending order behind those of the warps and blocks before it.  Bound by
// latency: up to five exchanges between blocks, or, for a block that is alone (up to 2048
// tokens), its own barriers and the clearing of its counters.  (Digits of 11 bits, one exchange less, took twice as long:
// the counts of eight blocks are then 64 KB a block and exchange.)  Measured with the move:
// 16 heads of 700 tokens 9.0 us, 32 heads from 32K to 1024 tokens 21 us.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBlockTokens = 2048;  // a block more for so many tokens, up to 8
constexpr int kSelCluster = 8;
// Keys of a slice kept in shared memory.  The launch goes by the capacity, which the lengths
// may be far below: where a full slice would not fit, there is room for the keys of shorter
// ones that costs no resident block (32 heads of 400,000 tokens to 1024: 190 us; with room
// for the most, one block a multiprocessor, 480).
constexpr int kSelSmemTokens = 40960, kSelSmemSome = 10240;
constexpr int kSelBins = 256;
constexpr int kSelCopies = 8;          // counters of a digit, by lane, as lanes often agree

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t sm_key[];
  __shared__ uint32_t hist[kSelBins * kSelCopies];
  __shared__ uint32_t total[2][kSelBins];  // of even and odd digits: a peer may still read the last one's
  __shared__ uint32_t sums[kSelBins];      // the cluster's counts
  __shared__ uint32_t s_digit, s_above, s_all;
  __shared__ int s_count[2];          // this block's tokens above the k-th key, and equal to it
  __shared__ int wsum[2][kSelWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x / C, b = hk / p.Hkv;
  grid_launch_dependents();  // the moving kernel's blocks come in while the last of these are at work
  bool badlen = false;
  const int len = (int)clamp_len(p.seq_lens[b], p.geo.Nmax, badlen);
  const int k = p.keep < len ? p.keep : len;
  if (tid == 0 && rank == 0) {
    if (badlen) atomicOr(p.err, kErrSeqLen);
    if (hk % p.Hkv == 0) p.new_lens[b] = k;
  }
  int32_t* kept = p.kept + (int64_t)hk * p.keep;
  for (int j = k + rank * kSelThreads + tid; j < p.keep; j += C * kSelThreads) kept[j] = -1;
  // (k is the same in the whole cluster: it leaves together)
  if (k == len) {  // everything stays
    for (int j = rank * kSelThreads + tid; j < k; j += C * kSelThreads) kept[j] = j;
    return;
  }
  if (k == 0) return;
  const float* mass = p.mass + (int64_t)hk * p.geo.Nmax;
  const int64_t recent0 = (int64_t)len - p.n_recent;
  // the block's slice, in runs of whole warps' loads so that every warp has one run
  const int t0 = (int)((int64_t)rank * len / C), t1 = (int)((int64_t)(rank + 1) * len / C);
  const bool in_smem = t1 - t0 <= p.smem_keys;
  auto global_key = [&](int t) { return t < p.n_sink || t >= recent0 ? 0xFFFFFFFFu : mass_key(mass[t]); };
  if (in_smem) {
    for (int t = t0 + tid; t < t1; t += kSelThreads) sm_key[t - t0] = global_key(t);
    __syncthreads();
  }
  auto key = [&](int t) { return in_smem ? sm_key[t - t0] : global_key(t); };

  uint32_t prefix = 0, mask = 0;
  int need = k;  // of the tokens whose digits so far equal prefix, this many are kept
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kSelBins * kSelCopies; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int t = t0 + tid; t < t1; t += kSelThreads) {
      const uint32_t u = key(t);
      if ((u & mask) == prefix) atomicAdd(&hist[((u >> shift) & 255) * kSelCopies + (lane & (kSelCopies - 1))], 1u);
    }
    __syncthreads();
    uint32_t* mine = total[(shift >> 3) & 1];
    if (tid < kSelBins) {
      uint32_t s = 0;
#pragma unroll
      for (int c = 0; c < kSelCopies; ++c) s += hist[tid * kSelCopies + c];
      mine[tid] = s;
      if (C == 1) sums[tid] = s;
    }
    if (C > 1) {
      cluster.sync();
      if (tid < kSelBins) {
        uint32_t s = 0;
#pragma unroll
        for (int c = 0; c < kSelCluster; ++c)
          if (c < C) s += cluster.map_shared_rank(mine, c)[tid];
        sums[tid] = s;
      }
    }
    __syncthreads();
    if (warp == 0) {
      // lane l: digits 255 - 8 l down to 248 - 8 l
      uint32_t d[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = sums[255 - 8 * lane - i];
        sum += d[i];
      }
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == __ffs(__ballot_sync(0xffffffffu, inc >= (uint32_t)need)) - 1) {
        uint32_t above = inc - sum, found = 0, at = 7, before = 0;
#pragma unroll
        for (int i = 7; i >= 0; --i) {  // the first i whose running count reaches need
          uint32_t run = above;
#pragma unroll
          for (int j = 0; j < 8; ++j) run += j < i ? d[j] : 0;
          if (run + d[i] >= (uint32_t)need) {
            at = i;
            before = run;
            found = d[i];
          }
        }
        s_digit = 255 - 8 * lane - at;
        s_above = before;
        s_all = before + found == (uint32_t)need;
      }
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    need -= (int)s_above;
    if (s_all) break;  // every key under these digits is kept
  }

  // kept: (key & mask) > prefix, and the first `need` that equal it; each warp has a run of tokens
  const int run = ((t1 - t0 + kSelThreads - 1) / kSelThreads) * 32;
  const int w0 = t0 + warp * run, w1 = w0 + run < t1 ? w0 + run : t1;
  int gt = 0, eq = 0;
  for (int t = w0 + lane; t < w1; t += 32) {
    const uint32_t u = key(t) & mask;
    gt += u > prefix;
    eq += u == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    wsum[0][warp] = gt;
    wsum[1][warp] = eq;
  }
  __syncthreads();
  if (tid < 2) {
    int s = 0;
    for (int w = 0; w < kSelWarps; ++w) s += wsum[tid][w];
    s_count[tid] = s;
  }
  cluster.sync();
  int base = 0, ties = 0;  // tokens above and ties before this warp's run
  for (int c = 0; c < rank; ++c) {
    const int* s = cluster.map_shared_rank(s_count, c);
    base += s[0];
    ties += s[1];
  }
  for (int w = 0; w < warp; ++w) {
    base += wsum[0][w];
    ties += wsum[1][w];
  }
  const uint32_t lt = (1u << lane) - 1u;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const uint32_t u = t < w1 ? key(t) & mask : 0u;
    const bool g = t < w1 && u > prefix, e = t < w1 && u == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
    const int te = ties + __popc(be & lt);  // ties before this token: the first `need` of them are kept
    if (g || (e && te < need)) kept[base + __popc(bg & lt) + (te < need ? te : need)] = t;
    base += __popc(bg);
    ties += __popc(be);
  }
  cluster.sync();  // the blocks' shared memory stays until every peer has read it
}

// ---------------------------------------------------------------- the kept rows move
// A warp moves groups of four tokens: 16 lanes a token's K row and 16 its V row, 16 bytes
// a lane; eight lanes the four code rows; four lanes the masses.
struct MoveGroup {
  uint4 kv[4], code;
  float mass;
};

// Sources (or destinations) of the group's tokens: lane j < 4 has token j's row number.
template <bool LOAD>
__device__ __forceinline__ void move_group(MoveGroup& m, const EvictParams& p, int64_t row, int cnt, int slot, int hk,
                                           int lane) {
  const uint16_t* kv = LOAD ? (lane < 16 ? p.K : p.V) : (lane < 16 ? p.K_out : p.V_out);
  const uint8_t* codes = LOAD ? p.codes : p.codes_out;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t r = __shfl_sync(0xffffffffu, row, j);
    if (j < cnt && r >= 0) {
      uint4* at = reinterpret_cast<uint4*>(const_cast<uint16_t*>(kv) + r * kDim) + (lane & 15);
      if (LOAD) m.kv[j] = *at;
      else *at = m.kv[j];
    }
  }
  if (p.codes) {
    const int64_t r = __shfl_sync(0xffffffffu, row, (lane >> 1) & 3);
    if (lane < 2 * cnt && r >= 0) {
      uint4* at = reinterpret_cast<uint4*>(const_cast<uint8_t*>(codes) + r * kCodeBytes) + (lane & 1);
      if (LOAD) m.code = *at;
      else *at = m.code;
    }
  }
  if (lane < cnt) {
    if (LOAD) m.mass = p.mass[(int64_t)hk * p.geo.Nmax + slot];
    else p.mass_out[(int64_t)hk * p.out.Nmax + slot] = m.mass;
  }
}

// To another cache: any block may move any rows; each has a run of them.  A warp has one
// group of rows on its way and looks up where the next one is meanwhile; 32 such warps fill
// a multiprocessor (two groups at a time leave room for 24 and took 140 us where this takes
// 119).  Bound by HBM (2 x 548 bytes a token) and the chain slot - page - row.  Measured:
// 4 x 8 heads of up to 32K tokens to 16K, pages to pages, 119 us with the selection (580 MB:
// 4.9 TB/s, 0.74 of the copy rate).
constexpr int kMoveThreads = 256;
constexpr int kMoveBlocks = 4;  // a multiprocessor

__global__ void __launch_bounds__(kMoveThreads, kMoveBlocks) evict_copy_kernel(const EvictParams p, int blocks_per_head) {
  constexpr int kStep = kMoveThreads / 32 * 4;  // rows of a round of the block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = blockIdx.x / blocks_per_head, part = blockIdx.x - hk * blocks_per_head;
  const int b = hk / p.Hkv, h = hk - b * p.Hkv;
  bool bad = false;
  const int len = (int)clamp_len(p.seq_lens[b], p.geo.Nmax, bad);
  const int k = p.keep < len ? p.keep : len;
  bad = false;
  const int32_t* kept = p.kept + (int64_t)hk * p.keep;
  // the block's rows, whole groups but for the last
  const int groups = (int)(((int64_t)k + 3) / 4);
  int j = (int)((int64_t)groups * part / blocks_per_head) * 4 + warp * 4;
  const int64_t last = (int64_t)groups * (part + 1) / blocks_per_head * 4;
  const int end = last < k ? (int)last : k;
  float* mass_out = p.mass_out + (int64_t)hk * p.out.Nmax;
  for (int64_t t = (int64_t)k + part * kMoveThreads + threadIdx.x; t < p.out.Nmax;
       t += (int64_t)blocks_per_head * kMoveThreads)
    mass_out[t] = 0.0f;
  grid_dependency_wait();  // kept is there
  int64_t from, to;
  int slot;
  auto look_up = [&](int64_t j0) {
    from = to = -1;
    slot = 0;
    if (lane < 4 && j0 + lane < end) {
      bool bad_to = false;
      slot = kept[j0 + lane];
      from = p.geo.row(b, h, slot, bad);
      to = p.out.row(b, h, (int)j0 + lane, bad_to);
      if (bad_to) to = -1;  // nothing is written through a bad entry
      bad |= bad_to;
    }
  };
  look_up(j);
  for (; j < end; j += kStep) {
    MoveGroup m;
    const int cnt = end - j < 4 ? end - j : 4;
    const int64_t dst = to;
    move_group<true>(m, p, from, cnt, slot, hk, lane);
    look_up((int64_t)j + kStep);
    move_group<false>(m, p, dst, cnt, j + lane, hk, lane);
    if (end - j <= kStep) break;
  }
  if (bad) atomicOr(p.err, kErrTable);
}

// In place: a kept row's destination is at or before its source, so a window of rows may
// be written once it and every window before it have been read -- which the blocks of a
// head's cluster tell each other by a barrier per window, the next window's rows on their
// way meanwhile (their sources lie behind every destination so far).  Rows before the
// first evicted token stay where they are.
constexpr int kShiftThreads = 512;

__global__ void __launch_bounds__(kShiftThreads) evict_shift_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  constexpr int kWarps = kShiftThreads / 32;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = blockIdx.x / C, b = hk / p.Hkv, h = hk - b * p.Hkv;
  bool bad = false;
  const int len = (int)clamp_len(p.seq_lens[b], p.geo.Nmax, bad);
  const int k = p.keep < len ? p.keep : len;
  bad = false;
  const int32_t* kept = p.kept + (int64_t)hk * p.keep;
  grid_dependency_wait();  // kept is there
  int lo = 0, hi = k;  // the first j whose slot is not j: kept[j] - j never falls
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (kept[mid] == mid) lo = mid + 1;
    else hi = mid;
  }
  const int window = C * kWarps * 4;
  MoveGroup m[2];
  int64_t to[2];
  auto read = [&](int g, int j) {  // this warp's rows of the window at j
    const int cnt = k - j < 4 ? (k - j < 0 ? 0 : k - j) : 4;
    int64_t from = -1;
    int slot = 0;
    to[g] = -1;
    if (lane < cnt) {
      slot = kept[j + lane];
      from = p.geo.row(b, h, slot, bad);
      bool bad_to = false;
      to[g] = p.geo.row(b, h, j + lane, bad_to);
      if (bad_to) to[g] = -1;
      bad |= bad_to;
    }
    move_group<true>(m[g], p, from, cnt, slot, hk, lane);
  };
  auto write = [&](int g, int j) {
    move_group<false>(m[g], p, to[g], k - j < 4 ? (k - j < 0 ? 0 : k - j) : 4, j + lane, hk, lane);
  };
  const int mine = lo + (rank * kWarps + warp) * 4;
  if (lo < k) read(0, mine);
  for (int j0 = lo; j0 < k; j0 += 2 * window) {
    const int j = mine + (j0 - lo);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      cluster_arrive();  // this window is in registers (the arrival orders the loads before)
      if (j0 + (g + 1) * window < k) read(1 - g, j + (g + 1) * window);
      cluster_wait();
      if (j0 + g * window < k) write(g, j + g * window);
    }
  }
  cluster.sync();  // every mass has moved
  float* mass_out = p.mass_out + (int64_t)hk * p.out.Nmax;
  for (int64_t t = k + rank * kShiftThreads + threadIdx.x; t < p.out.Nmax; t += (int64_t)C * kShiftThreads)
    mass_out[t] = 0.0f;
  if (bad) atomicOr(p.err, kErrTable);
}

}  // namespace adamas
