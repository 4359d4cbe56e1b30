// Rotary positions of new q and k rows, and the append of the new rows (and of the
// rotated keys' codes) to the cache.
//
// Pair (x1, x2) of a row at position p turns by the angle 2 pi frac(f p):
//   x1' = x1 c - x2 s,  x2' = x2 c + x1 s,  c = m cos, s = m sin.
// f is kept as a 64-bit fraction of a turn, so the 64-bit product f p drops whole
// turns by itself and the angle of position 10^6 is as exact as that of position 1
// (an fp32 angle there is off by 0.06 rad).  cos and sin are evaluated in 64 bits
// once per (token, pair) -- 64 evaluations for 40 and more heads -- and rounded to
// fp32; the products and the sum are rounded to fp32 one by one, without a fused
// multiply-add, so that the rotated keys, and the codes made from them, are the same
// bits wherever they are computed this way.
#pragma once

#include "cache.cuh"
#include "encode.cuh"

namespace adamas {

struct RopeParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *cu_new, *cache_lens, *positions;
  const uint64_t* freqs;
  int rot, interleaved;
  double mscale;
  int T, B, Hq, Hkv;
  uint16_t* q_out;
  uint16_t *K, *V;
  uint8_t* codes;
  CacheGeom geo;
  uint32_t* err;
};

constexpr int kRopeThreads = 256;

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The lane's four elements 4 lane .. 4 lane + 3 of a row, rotated.  cs holds (c, s)
// of every pair; x is the row (read again for partners that no single lane holds).
__device__ __forceinline__ uint2 rope_row(const uint16_t* x, uint2 raw, const float2* cs, int rot, int interleaved,
                                          int lane) {
  float v[4] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y)};
  float o[4];
  const int half = rot >> 1, e0 = 4 * lane;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      o[i] = v[i];
      o[i + 1] = v[i + 1];
      if (e0 + i < rot) {
        const float2 t = cs[(e0 + i) >> 1];
        o[i] = __fsub_rn(__fmul_rn(v[i], t.x), __fmul_rn(v[i + 1], t.y));
        o[i + 1] = __fadd_rn(__fmul_rn(v[i + 1], t.x), __fmul_rn(v[i], t.y));
      }
    }
  } else {
    float w[4];  // the partners
    if ((half & 3) == 0) {  // the partner of a lane's elements is one lane's elements
      const int d = half >> 2;
      const int src = e0 < half ? lane + d : lane - d;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __shfl_sync(0xffffffffu, v[i], src & 31);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = e0 + i, p = e < half ? e + half : e - half;
        w[i] = e < rot ? __uint_as_float((uint32_t)x[p] << 16) : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + i;
      o[i] = v[i];
      if (e < half) {
        const float2 t = cs[e];
        o[i] = __fsub_rn(__fmul_rn(v[i], t.x), __fmul_rn(w[i], t.y));
      } else if (e < rot) {
        const float2 t = cs[e - half];
        o[i] = __fadd_rn(__fmul_rn(v[i], t.x), __fmul_rn(w[i], t.y));
      }
    }
  }
  // unrotated elements keep their bits (a NaN's payload too)
  uint2 r = make_uint2(bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]));
  if (e0 >= rot) r.x = raw.x;
  if (e0 + 2 >= rot) r.y = raw.y;
  return r;
}

// One block per token (grid.x) and share of its rows (grid.y): the block's threads
// evaluate the token's cos and sin, then each warp takes rows of the Hq query heads,
// the Hkv keys and the Hkv values in turn.
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p) {
  __shared__ float2 cs[kDim / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x;
  // the sequence of row r: the last one that starts at or before it
  int below = 0;
  for (int b0 = 0; b0 < p.B; b0 += kRopeThreads)
    below += __syncthreads_count(b0 + tid < p.B && p.cu_new[b0 + tid] <= r);
  const int b = below - 1;
  if (b < 0) return;  // a row before the first sequence
  int first, n;
  bool bad = false;
  ragged_rows(p.cu_new, b, p.T, first, n, bad);
  if (bad && p.err && tid == 0) atomicOr(p.err, kErrOffsets);
  if (r < first || r >= first + n) return;  // behind the last sequence
  const int64_t slot64 = (int64_t)p.cache_lens[b] + (r - first);
  const int pos = p.positions ? p.positions[r] : (int)slot64;
  if (tid < p.rot / 2) {
    const uint64_t turn = p.freqs[tid] * (uint64_t)(int64_t)pos;
    double s, c;
    sincospi((double)(int64_t)turn * 0x1p-63, &s, &c);
    cs[tid] = make_float2((float)(c * p.mscale), (float)(s * p.mscale));
  }
  __syncthreads();
  const int nq = p.q ? p.Hq : 0, nk = p.k ? p.Hkv : 0;
  const bool in_cache = slot64 >= 0 && slot64 < p.geo.Nmax;
  const int rows = nq + 2 * nk;
  for (int i = blockIdx.y * (kRopeThreads / 32) + warp; i < rows; i += gridDim.y * (kRopeThreads / 32)) {
    const bool is_q = i < nq, is_k = !is_q && i < nq + nk;
    const int h = is_q ? i : (is_k ? i - nq : i - nq - nk);
    const uint16_t* x = is_q ? p.q + r * p.q_stride : (is_k ? p.k + r * p.k_stride : p.v + r * p.v_stride);
    x += h * kDim;
    if (!is_q && !in_cache) continue;
    const uint2 raw = *reinterpret_cast<const uint2*>(x + 4 * lane);
    uint2 o = raw;
    if (is_q || is_k) o = rope_row(x, raw, cs, p.rot, p.interleaved, lane);
    __syncwarp();  // every lane has read the row: q_out may be q
    if (is_q) {
      *reinterpret_cast<uint2*>(p.q_out + ((int64_t)r * p.Hq + h) * kDim + 4 * lane) = o;
      continue;
    }
    bool bad_page = false;
    const int64_t row = p.geo.row(b, h, (int)slot64, bad_page);
    if (bad_page) {
      if (p.err && lane == 0) atomicOr(p.err, kErrTable);
      continue;
    }
    *reinterpret_cast<uint2*>((is_k ? p.K : p.V) + row * kDim + 4 * lane) = o;
    if (is_k && p.codes) {
      const uint32_t w = encode128_warp_raw(o, lane);
      if (lane < kCodeWords) reinterpret_cast<uint32_t*>(p.codes + row * kCodeBytes)[lane] = w;
    }
  }
}

}  // namespace adamas
