// Attention weight of the decode step's kept tokens, and the eviction of the tokens
// with the least accumulated weight.
#pragma once

#include "cache.cuh"
#include "chunk.cuh"

namespace adamas {

struct KeptParams {
  const uint16_t *q, *K;
  const int32_t *idx, *seq_lens;
  int B, Hq, Hkv, G, budget, shared_rows;
  float* mass;
  CacheGeom geo;
  uint32_t* err;
};

// One block per (b, kv head); its query heads one after the other, so that the
// weights of two heads that kept the same token are added in a fixed order.
__global__ void __launch_bounds__(256) accumulate_kept_kernel(const KeptParams p) {
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
  CacheGeom geo, out;
  uint32_t* err;
};

constexpr int kSelThreads = 1024;

// Order-preserving image of a mass in unsigned integers: larger is kept first.  -0 is
// 0; NaN is below everything; forced tokens are above everything.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One block per (b, kv head): the k-th largest key by four 8-bit digits (most
// significant first), then the kept slots in ascending order.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_digit, s_above;
  __shared__ int wsum[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x, b = hk / p.Hkv;
  bool badlen = false;
  const int len = (int)clamp_len(p.seq_lens[b], p.geo.Nmax, badlen);
  const int k = p.keep < len ? p.keep : len;
  if (tid == 0) {
    if (badlen) atomicOr(p.err, kErrSeqLen);
    if (hk % p.Hkv == 0) p.new_lens[b] = k;
  }
  int32_t* kept = p.kept + (int64_t)hk * p.keep;
  for (int j = k + tid; j < p.keep; j += kSelThreads) kept[j] = -1;
  if (k == 0) return;
  const float* mass = p.mass + (int64_t)hk * p.geo.Nmax;
  const int64_t recent0 = (int64_t)len - p.n_recent;
  auto key = [&](int t) { return t < p.n_sink || t >= recent0 ? 0xFFFFFFFFu : mass_key(mass[t]); };
  uint32_t prefix = 0, mask = 0;
  int need = k;  // of the tokens whose digits so far equal prefix, this many are kept
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int t = tid; t < len; t += kSelThreads) {
      const uint32_t u = key(t);
      if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t above = 0;
      int d = 255;
      while (d > 0 && above + hist[d] < (uint32_t)need) above += hist[d--];
      s_digit = d;
      s_above = above;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    need -= (int)s_above;
    __syncthreads();
  }
  // kept: key > prefix, and the first `need` of key == prefix
  int base = 0, ties = 0;
  for (int t0 = 0; t0 < len; t0 += kSelThreads) {
    const int t = t0 + tid;
    const uint32_t u = t < len ? key(t) : 0u;
    const bool gt = t < len && u > prefix, eq = t < len && u == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      wsum[0][warp] = __popc(bg);
      wsum[1][warp] = __popc(be);
    }
    __syncthreads();
    int g0 = 0, e0 = 0, gall = 0, eall = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) g0 += wsum[0][w], e0 += wsum[1][w];
      gall += wsum[0][w], eall += wsum[1][w];
    }
    const uint32_t lt = (1u << lane) - 1u;
    const int te = ties + e0 + __popc(be & lt);        // ties before this token
    const int pos = base + g0 + __popc(bg & lt) + (te - ties < need - ties ? te - ties : (need - ties > 0 ? need - ties : 0));
    if (gt || (eq && te < need)) kept[pos] = t;
    const int tk = need - ties < 0 ? 0 : (need - ties < eall ? need - ties : eall);
    base += gall + tk;
    ties += eall;
    __syncthreads();
  }
}

// The kept rows of one (b, kv head), moved in order.  In place a row's destination is
// at or before its source, so a window of rows is read before any of it is written.
constexpr int kMoveThreads = 1024;
constexpr int kMoveChunks = 34;  // 16-byte pieces of a token: 16 of K, 16 of V, 2 of codes

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  constexpr int kRows = 120;  // rows of a window: 4 pieces a thread
  const int tid = threadIdx.x;
  const int hk = blockIdx.x, b = hk / p.Hkv, h = hk - b * p.Hkv;
  bool bad = false;
  const int len = (int)clamp_len(p.seq_lens[b], p.geo.Nmax, bad);
  const int k = p.keep < len ? p.keep : len;
  bad = false;
  const int32_t* kept = p.kept + (int64_t)hk * p.keep;
  const float* mass = p.mass + (int64_t)hk * p.geo.Nmax;
  float* mass_out = p.mass_out + (int64_t)hk * p.out.Nmax;
  for (int j0 = 0; j0 < k; j0 += kRows) {
    uint4 w[4];
    uint4* dst[4];
    float mv = 0.0f;
    const int rows = k - j0 < kRows ? k - j0 : kRows;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = tid + i * kMoveThreads;
      dst[i] = nullptr;
      if (c < rows * kMoveChunks) {
        const int j = j0 + c / kMoveChunks, piece = c % kMoveChunks;
        bool bad_src = false, bad_dst = false;
        const int64_t rs = p.geo.row(b, h, kept[j], bad_src), rd = p.out.row(b, h, j, bad_dst);
        bad |= bad_src || bad_dst;
        const bool code = piece >= 32;
        if (!bad_dst && (!code || p.codes)) {
          const unsigned char* s = code ? p.codes + rs * kCodeBytes + (piece - 32) * 16
                                        : reinterpret_cast<const unsigned char*>((piece < 16 ? p.K : p.V) + rs * kDim) + (piece & 15) * 16;
          unsigned char* d = code ? p.codes_out + rd * kCodeBytes + (piece - 32) * 16
                                  : reinterpret_cast<unsigned char*>((piece < 16 ? p.K_out : p.V_out) + rd * kDim) + (piece & 15) * 16;
          w[i] = *reinterpret_cast<const uint4*>(s);
          dst[i] = reinterpret_cast<uint4*>(d);
        }
      }
    }
    if (tid < rows) mv = mass[kept[j0 + tid]];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (dst[i]) *dst[i] = w[i];
    if (tid < rows) mass_out[j0 + tid] = mv;
    __syncthreads();
  }
  for (int64_t t = k + tid; t < p.out.Nmax; t += kMoveThreads) mass_out[t] = 0.0f;
  if (bad) atomicOr(p.err, kErrTable);
}

}  // namespace adamas
