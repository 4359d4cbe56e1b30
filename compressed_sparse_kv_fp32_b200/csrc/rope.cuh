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
  int rot;
  double mscale;
  int T, B, Hq, Hkv;
  int tokens;  // of a block
  uint16_t* q_out;
  uint16_t *K, *V;
  uint8_t* codes;
  CacheGeom geo;
  uint32_t* err;
  uint64_t neg0;  // -0 twice
};

constexpr int kRopeThreads = 128;

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sixteen lanes hold a row, eight elements 8 l .. 8 l + 7 each, so that a warp has two
// rows in hand.  How a lane gets its elements' partners:
constexpr int kRopeShuffle = 0;  // half layout, rot % 16 == 0: they are one other lane's elements
constexpr int kRopeInside = 1;   // interleaved: its own
constexpr int kRopeLoad = 2;     // half layout, other rot: read from the row again

__device__ __forceinline__ uint64_t bf16_to_f2(uint32_t w) { return f2_pack(bf16_lo(w), bf16_hi(w)); }

// What a lane needs of its token, the same for every row: cos and signed sin of its
// elements in pairs (x' = x c + partner s with s negative for the first of a rotated pair:
// the product's sign is exact, so this is the difference of the definition bit for bit).
struct RopeLane {
  uint64_t c[4], s[4];
  // A packed multiplication followed by a packed addition came out as one fused operation,
  // whose result can be a rounding off.  Here a product is a fused operation with a -0
  // that the compiler does not know: the rounded product, and not to be merged.
  uint64_t neg0;
  uint32_t on;  // bit i: elements 2 i and 2 i + 1 are rotated
};

template <int MODE>
__device__ __forceinline__ uint4 rope_row(const uint16_t* x, uint4 raw, const RopeLane& t, int partner, int rot, int l) {
  const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t w;
    if constexpr (MODE == kRopeShuffle) {
      w = bf16_to_f2(__shfl_sync(0xffffffffu, v[i], partner));
    } else if constexpr (MODE == kRopeInside) {
      w = f2_pack(bf16_hi(v[i]), bf16_lo(v[i]));
    } else {
      const int e = 8 * l + 2 * i, half = rot >> 1;
      float a = 0.0f, b = 0.0f;
      if (e < rot) {  // rot is even: the pair is rotated or not
        a = __uint_as_float((uint32_t)x[e < half ? e + half : e - half] << 16);
        b = __uint_as_float((uint32_t)x[e + 1 < half ? e + 1 + half : e + 1 - half] << 16);
      }
      w = f2_pack(a, b);
    }
    float a, b;
    f2_unpack(f2_add(f2_fma(bf16_to_f2(v[i]), t.c[i], t.neg0), f2_fma(w, t.s[i], t.neg0)), a, b);
    // unrotated elements keep their bits (a NaN's payload too)
    o[i] = t.on >> i & 1 ? bf16_pair(a, b) : v[i];
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The 2-bit codes of the row in each half of a warp: the arithmetic of encode128_warp
// (stage h pairs elements h apart, ascending; then one multiplication), stages 1, 2, 4
// inside a lane, 8 .. 64 between lanes.  Returns the lane's eight codes in 16 bits, in
// the order of the packed bytes.
__device__ __forceinline__ uint32_t encode128_half(uint4 raw, int l) {
  float v[8] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y),
                bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w)};
#pragma unroll
  for (int h = 1; h < 8; h *= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & h)) {
        const float a = v[i], b = v[i + h];
        v[i] = __fadd_rn(a, b);
        v[i + h] = __fsub_rn(a, b);
      }
#pragma unroll
  for (int m = 1; m < 16; m *= 2) {  // h = 8 m: the upper lane holds x[j + h] and gets x[j] - x[j + h]
    const bool upper = (l & m) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __shfl_xor_sync(0xffffffffu, v[i], m);
      v[i] = __fadd_rn(q, upper ? -v[i] : v[i]);  // the same as q - v and, addition commuting, v + q
    }
  }
  const float c = hadamard_norm();
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = __fmul_rn(v[i], c);
    mx = fmaxf(mx, fabsf(v[i]));
  }
#pragma unroll
  for (int m = 8; m > 0; m /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
  const float t0 = -0.5f * mx, t2 = 0.5f * mx;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= code_of(v[i], t0, t2) << ((i < 4 ? 6 : 14) - 2 * (i & 3));
  return w;
}

// A block has kRopeTokens tokens, two warps each, or, when there are few tokens, one, whose
// rows may be shared by several blocks (grid.y).  While a warp's first rows (of the Hq
// query heads, the Hkv keys and the Hkv values in turn, two at a time) are on their way,
// two warps per token find its sequence and place and evaluate its cos and sin; a row's
// registers are asked for again as soon as it is done.  Bound by instructions and HBM
// when there are many tokens, by latency for a few.  Measured: 12,506 tokens of 32 + 2 x 8
// heads with codes 74 us (4.2 TB/s, 0.64 of the copy rate), one token of 32 + 2 x 32 heads
// 3.4 us.  (One row a warp, every lane asking which half it holds: 229 us; cos and signed
// sin kept per lane: 115; two rows a warp on packed pairs and two warps a token: 79;
// seven blocks of 128 threads a multiprocessor, whose 72 registers a thread are enough, for
// four of 256 that kept some in memory: 74.)
constexpr int kRopeAhead = 4;  // pairs of rows
constexpr int kRopeTokens = kRopeThreads / 64;

template <int MODE>
__global__ void __launch_bounds__(kRopeThreads, 7) rope_append_kernel(const RopeParams p) {
  __shared__ float2 cs[kRopeTokens][kDim / 2];
  __shared__ int64_t row0_of[kRopeTokens];  // its row in the cache's first head; -1: in no sequence, -2: not stored
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 15, hi = lane >> 4, e0 = 8 * l;
  const int nq = p.q ? p.Hq : 0, nk = p.k ? p.Hkv : 0, rows = nq + 2 * nk, pairs = (rows + 1) >> 1;
  const int share = (kRopeThreads / 32) / p.tokens;  // warps of a token: 4 or 2
  const int tk = warp / share, part = warp - tk * share;
  const int64_t r = (int64_t)blockIdx.x * p.tokens + tk;
  const int stride = gridDim.y * share, i0 = r < p.T ? blockIdx.y * share + part : pairs;

  auto source = [&](int i) {
    return (i < nq ? p.q + r * p.q_stride + i * kDim
                   : (i < nq + nk ? p.k + r * p.k_stride + (i - nq) * kDim
                                  : p.v + r * p.v_stride + (i - nq - nk) * kDim)) + e0;
  };
  auto ask = [&](int pair) {
    const int i = 2 * pair + hi;
    return i < rows ? *reinterpret_cast<const uint4*>(source(i)) : make_uint4(0, 0, 0, 0);
  };
  uint4 raw[kRopeAhead];
#pragma unroll
  for (int j = 0; j < kRopeAhead; ++j) raw[j] = ask(i0 + j * stride);

  if (blockIdx.x == 0 && blockIdx.y == 0) {  // the offsets of sequences that no row is looked up in, too
    bool bad = false;
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += kRopeThreads) {
      int first, n;
      ragged_rows(p.cu_new, b, p.T, first, n, bad);
    }
    if (bad) atomicOr(p.err, kErrOffsets);
  }
  if (part < 2 && r < p.T) {
    int below = 0;  // the sequence of row r is the last one that starts at or before it
    for (int b0 = 0; b0 < p.B; b0 += 32)
      below += __popc(__ballot_sync(0xffffffffu, b0 + lane < p.B && p.cu_new[b0 + lane] <= r));
    int64_t row0 = -1;
    if (below > 0) {
      int first, n;
      bool bad = false;  // flagged above
      ragged_rows(p.cu_new, below - 1, p.T, first, n, bad);
      if (r >= first && r < first + n) {
        const int64_t slot = (int64_t)p.cache_lens[below - 1] + (r - first);
        const int pair = part * 32 + lane;
        if (pair < p.rot / 2) {
          const int64_t pos = p.positions ? p.positions[r] : slot;
          const uint64_t turn = p.freqs[pair] * (uint64_t)pos;
          double s, c;
          sincospi((double)(int64_t)turn * 0x1p-63, &s, &c);
          cs[tk][pair] = make_float2((float)(c * p.mscale), (float)(s * p.mscale));
        }
        row0 = -2;
        if (nk && slot >= 0 && slot < p.geo.Nmax) {
          bool bad_page = false;
          const int64_t row = p.geo.row(below - 1, 0, (int)slot, bad_page);
          if (!bad_page) row0 = row;
          else if (lane == 0) atomicOr(p.err, kErrTable);
        }
      }
    }
    if (part == 0 && lane == 0) row0_of[tk] = row0;
  }
  __syncthreads();
  if (i0 >= pairs) return;
  const int64_t row0 = row0_of[tk];
  if (row0 == -1) return;
  const int64_t head_rows = p.geo.table ? p.geo.page.d : p.geo.Nmax;  // from one head's row to the next one's
  const int half = p.rot >> 1;
  const int partner = (e0 < half ? lane + (half >> 3) : lane - (half >> 3)) & 31;
  RopeLane t;
  t.on = 0;
  t.neg0 = p.neg0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float c[2], s[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int e = e0 + 2 * k + m;
      const bool second = MODE == kRopeInside ? m : e >= half;
      const float2 z = e < p.rot ? cs[tk][MODE == kRopeInside ? e >> 1 : (second ? e - half : e)] : make_float2(1.0f, 0.0f);
      c[m] = z.x;
      s[m] = second ? z.y : -z.y;
    }
    t.c[k] = f2_pack(c[0], c[1]);
    t.s[k] = f2_pack(s[0], s[1]);
    t.on |= (uint32_t)(e0 + 2 * k < p.rot) << k;
  }
  for (int p0 = i0; p0 < pairs; p0 += kRopeAhead * stride) {
#pragma unroll
    for (int j = 0; j < kRopeAhead; ++j) {
      const int pair = p0 + j * stride, i = 2 * pair + hi;
      if (pair >= pairs) break;
      const uint4 in = raw[j];
      const bool rotate = i < nq + nk, some = 2 * pair < nq + nk;
      uint4 o = in;
      if (some) {
        o = rope_row<MODE>(MODE == kRopeLoad ? source(rotate ? i : 2 * pair) - e0 : nullptr, in, t, partner, p.rot, l);
        if (!rotate) o = in;
        if (MODE == kRopeLoad) __syncwarp();  // every lane has read the row: q_out may be q
      }
      if (p0 + kRopeAhead * stride < pairs) raw[j] = ask(pair + kRopeAhead * stride);
      if (i < nq) {
        *reinterpret_cast<uint4*>(p.q_out + (r * p.Hq + i) * kDim + e0) = o;
      } else if (row0 >= 0 && i < rows) {
        const int64_t row = row0 + (rotate ? i - nq : i - nq - nk) * head_rows;
        *reinterpret_cast<uint4*>((rotate ? p.K : p.V) + row * kDim + e0) = o;
      }
      if (p.codes && some && 2 * pair + 1 >= nq && row0 >= 0) {  // a key among the two rows
        uint32_t w = encode128_half(o, l);
        w |= __shfl_down_sync(0xffffffffu, w, 1) << 16;
        if (i >= nq && rotate && (l & 1) == 0)
          reinterpret_cast<uint32_t*>(p.codes + (row0 + (i - nq) * head_rows) * kCodeBytes)[l >> 1] = w;
      }
    }
  }
}

}  // namespace adamas
