// Causal attention of a ragged chunk of new tokens over the cache, and the
// attention weight each cached token received from it.
#pragma once

#include "cache.cuh"

namespace adamas {

struct ChunkParams {
  const uint16_t *q, *K, *V;
  const int32_t *cu_q, *seq_lens;
  int T, B, Hq, Hkv, G;
  uint16_t* out;
  float* lse;
  float* mass;
  CacheGeom geo;
  uint32_t* err;
};

constexpr float kScoreScale = 0.08838834764831845f;               // 1 / sqrt(128)
constexpr float kScoreLog2 = 0.08838834764831845f * 1.4426950408889634f;  // ... log2 e

// sequence of packed row r (-1: none), found by every warp on its own
__device__ __forceinline__ int sequence_of_row(const int32_t* cu, int B, int T, int r, int lane, int& first, int& n,
                                               bool& bad) {
  int below = 0;
  for (int b0 = 0; b0 < B; b0 += 32)
    below += __popc(__ballot_sync(0xffffffffu, b0 + lane < B && cu[b0 + lane] <= r));
  if (below == 0) return -1;
  ragged_rows(cu, below - 1, T, first, n, bad);
  return r >= first && r < first + n ? below - 1 : -1;
}

// One warp per (row, query head): groups of 32 slots, a lane's score each, then the
// lanes' four output dimensions over the group.
__global__ void __launch_bounds__(128) chunk_attend_rows_kernel(const ChunkParams p) {
  __shared__ float sq[4][kDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = (int64_t)blockIdx.x * 4 + warp;
  if (item >= (int64_t)p.T * p.Hq) return;
  const int r = (int)(item / p.Hq), h = (int)(item - (int64_t)r * p.Hq), kvh = h / p.G;
  int first = 0, n = 0;
  bool bad = false, badlen = false, badpage = false;
  const int b = sequence_of_row(p.cu_q, p.B, p.T, r, lane, first, n, bad);
  if (bad && lane == 0) atomicOr(p.err, kErrOffsets);
  if (b < 0) return;
  const int64_t len = clamp_len(p.seq_lens[b], p.geo.Nmax, badlen);
  if (badlen && lane == 0) atomicOr(p.err, kErrSeqLen);
  const int64_t at = len - n + (r - first);
  const uint2 raw = *reinterpret_cast<const uint2*>(p.q + item * kDim + 4 * lane);
  sq[warp][4 * lane] = bf16_lo(raw.x);
  sq[warp][4 * lane + 1] = bf16_hi(raw.x);
  sq[warp][4 * lane + 2] = bf16_lo(raw.y);
  sq[warp][4 * lane + 3] = bf16_hi(raw.y);
  __syncwarp();
  float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
  for (int t0 = 0; t0 <= at; t0 += 32) {
    const int t = t0 + lane;
    float s = -INFINITY;
    int64_t row = 0;
    if (t <= at) {
      row = p.geo.row(b, kvh, t, badpage);
      const uint4* k = reinterpret_cast<const uint4*>(p.K + row * kDim);
      float a = 0.0f;
      for (int c = 0; c < 16; ++c) {
        const uint4 w = k[c];
        const float* qq = &sq[warp][8 * c];
        a += qq[0] * bf16_lo(w.x) + qq[1] * bf16_hi(w.x) + qq[2] * bf16_lo(w.y) + qq[3] * bf16_hi(w.y) +
             qq[4] * bf16_lo(w.z) + qq[5] * bf16_hi(w.z) + qq[6] * bf16_lo(w.w) + qq[7] * bf16_hi(w.w);
      }
      s = a * kScoreLog2;
    }
    float mx = s;
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float mn = fmaxf(m, mx), f = exp2f(m - mn), e = exp2f(s - mn);
    float sum = e;
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * f + sum;
    m = mn;
    for (int i = 0; i < 4; ++i) o[i] *= f;
    const int cnt = at - t0 + 1 < 32 ? (int)(at - t0 + 1) : 32;
    for (int j = 0; j < cnt; ++j) {
      const float w = __shfl_sync(0xffffffffu, e, j);
      const int64_t rj = __shfl_sync(0xffffffffu, row, j);
      const uint2 v = *reinterpret_cast<const uint2*>(p.V + rj * kDim + 4 * lane);
      o[0] += w * bf16_lo(v.x);
      o[1] += w * bf16_hi(v.x);
      o[2] += w * bf16_lo(v.y);
      o[3] += w * bf16_hi(v.y);
    }
  }
  if (badpage) atomicOr(p.err, kErrTable);
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint32_t w0, w1;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w0) : "f"(o[1] * inv), "f"(o[0] * inv));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w1) : "f"(o[3] * inv), "f"(o[2] * inv));
  *reinterpret_cast<uint2*>(p.out + item * kDim + 4 * lane) = make_uint2(w0, w1);
  if (p.lse && lane == 0) p.lse[item] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// One thread per slot: its key in registers, the chunk's rows one after the other.
__global__ void __launch_bounds__(128) accumulate_chunk_rows_kernel(const ChunkParams p) {
  __shared__ float sq[kDim];
  const int tid = threadIdx.x;
  const int hk = blockIdx.y, b = hk / p.Hkv, kvh = hk - b * p.Hkv;
  int first, n;
  bool bad = false, badlen = false, badpage = false;
  ragged_rows(p.cu_q, b, p.T, first, n, bad);
  const int64_t len = clamp_len(p.seq_lens[b], p.geo.Nmax, badlen);
  if (tid == 0 && bad) atomicOr(p.err, kErrOffsets);
  if (tid == 0 && badlen) atomicOr(p.err, kErrSeqLen);
  const int64_t t = (int64_t)blockIdx.x * 128 + tid;
  if ((int64_t)blockIdx.x * 128 >= len || n == 0) return;
  uint4 k[16] = {};
  if (t < len) {
    const int64_t row = p.geo.row(b, kvh, (int)t, badpage);
    for (int c = 0; c < 16; ++c) k[c] = reinterpret_cast<const uint4*>(p.K + row * kDim)[c];
  }
  if (badpage) atomicOr(p.err, kErrTable);
  float acc = 0.0f;
  for (int i = 0; i < n; ++i)
    for (int g = 0; g < p.G; ++g) {
      const int64_t item = (int64_t)(first + i) * p.Hq + kvh * p.G + g;
      __syncthreads();
      sq[tid] = __uint_as_float((uint32_t)p.q[item * kDim + tid] << 16);
      __syncthreads();
      const float z = p.lse[item];
      if (t >= len || t > len - n + i || z == -INFINITY) continue;
      float a = 0.0f;
      for (int c = 0; c < 16; ++c) {
        const uint4 w = k[c];
        const float* qq = &sq[8 * c];
        a += qq[0] * bf16_lo(w.x) + qq[1] * bf16_hi(w.x) + qq[2] * bf16_lo(w.y) + qq[3] * bf16_hi(w.y) +
             qq[4] * bf16_lo(w.z) + qq[5] * bf16_hi(w.z) + qq[6] * bf16_lo(w.w) + qq[7] * bf16_hi(w.w);
      }
      acc += expf(a * kScoreScale - z);
    }
  if (t < len) p.mass[(int64_t)hk * p.geo.Nmax + t] += acc;
}

}  // namespace adamas
