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
