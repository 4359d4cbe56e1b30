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

constexpr float kScoreLog2 = 0.08838834764831845f * 1.4426950408889634f;  // ... log2 e

}  // namespace adamas
