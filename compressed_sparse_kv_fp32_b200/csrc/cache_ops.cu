// C ABI of the cache operators (declared in include/adamas.h): rotary append, chunk
// attention, accumulated attention weights, eviction.  Argument checks and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/adamas.h"
#include "chunk_attend.cuh"
#include "chunk_weights.cuh"
#include "evict.cuh"
#include "rope.cuh"

namespace adamas {

int cuda_fail(cudaError_t e);  // adamas.cu: records the error, returns ADAMAS_ERR_CUDA

static_assert(kErrOffsets == ADAMAS_DEVERR_OFFSETS, "error bits of the header");

constexpr int kCopyBlocks = 148 * kMoveBlocks;  // as many as are resident: each then streams
constexpr int64_t kRopeSplitBlocks = 592;  // blocks up to which a token's rows are split: four a multiprocessor, of the seven that fit
constexpr size_t kCtrlBytes = 256;  // control words at the start of every workspace

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Sizes common to the operators (Hq = Hkv where a call has no query heads).
static int check_heads(int B, int Hq, int Hkv, int d) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return ADAMAS_ERR_INVALID_ARG;
  if (d != kDim) return ADAMAS_ERR_UNSUPPORTED;
  if (Hq / Hkv > kMaxGroup || B > kMaxBatch || (int64_t)B * Hkv > 65535) return ADAMAS_ERR_UNSUPPORTED;
  return ADAMAS_OK;
}

static int make_geom(const int32_t* table, int64_t n_pages, int page_size, int max_pages, int64_t Nmax, int Hkv,
                     CacheGeom* g) {
  g->table = table;
  g->Hkv = Hkv;
  g->Nmax = Nmax;
  g->n_pages = 0;
  g->max_pages = 0;
  if (table) {
    if (page_size < 1 || max_pages < 1 || n_pages < 1 || !aligned(table, 4)) return ADAMAS_ERR_INVALID_ARG;
    g->Nmax = (int64_t)max_pages * page_size;
    g->n_pages = n_pages;
    g->max_pages = max_pages;
    g->page = FastDiv::of((uint32_t)page_size);
  }
  if (g->Nmax < 0) return ADAMAS_ERR_INVALID_ARG;
  if (g->Nmax > INT32_MAX) return ADAMAS_ERR_UNSUPPORTED;
  return ADAMAS_OK;
}

static int check_ctrl(const void* ws, size_t bytes, size_t need) {
  return !ws || bytes < need || !aligned(ws, 16) ? ADAMAS_ERR_WORKSPACE : ADAMAS_OK;
}

static uint32_t* err_word(void* ws) { return static_cast<uint32_t*>(ws) + 2; }

// A launch in clusters of C blocks; `most` bytes of dynamic shared memory are allowed to
// the kernel once per device.  `early`: its blocks may come in before the launch in front of
// it is done (the kernel waits for that itself).
template <auto Kernel, typename... Args>
static int launch_cluster(int grid, int C, int threads, size_t smem, size_t most, bool early, cudaStream_t st,
                          Args... args) {
  cudaError_t e;
  if (most > 48 * 1024) {
    static std::atomic<uint64_t> known{0};  // a bit per device
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_fail(e);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(known.load(std::memory_order_acquire) & bit) || bit == 0) {
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(Kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
      if (e != cudaSuccess) return cuda_fail(e);
      known.fetch_or(bit, std::memory_order_release);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = early ? 2 : 1;
  if ((e = cudaLaunchKernelEx(&cfg, Kernel, args...)) != cudaSuccess) {
    (void)cudaGetLastError();
    return cuda_fail(e);
  }
  return ADAMAS_OK;
}

static int launched() {
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? cuda_fail(e) : ADAMAS_OK;
}

// Multiprocessors of the current device, with the one-time set-up of the chunk kernels on
// it: their shared memory, and the register count that chunk attention's split is made for.
static int attend_device(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= 64) return ADAMAS_ERR_UNSUPPORTED;
  if ((*sms = known[dev].load(std::memory_order_acquire)) > 0) return ADAMAS_OK;
  const void* fn = reinterpret_cast<const void*>(&chunk_attend_kernel);
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, fn)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAtSmem)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&chunk_weights_kernel),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWtSmem)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return cuda_fail(e);
  if (fa.numRegs != 65536 / kAtThreads) return ADAMAS_ERR_UNSUPPORTED;  // the warps' shares add up to 65536
  if (*sms > kAtMaxGrid) *sms = kAtMaxGrid;
  known[dev].store(*sms, std::memory_order_release);
  return ADAMAS_OK;
}

// Tensor maps of bf16 arrays for copies of 64 columns (128 bytes, the swizzle's width).  The
// encoder is a driver call, reached through the runtime.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static int tile_map(const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                    const cuuint32_t* boxes, CUtensorMap* map) {
  static std::atomic<EncodeTiledFn> known{nullptr};
  EncodeTiledFn fn = known.load(std::memory_order_acquire);
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return cuda_fail(e);
    if (q != cudaDriverEntryPointSuccess || !f) return ADAMAS_ERR_UNSUPPORTED;
    fn = reinterpret_cast<EncodeTiledFn>(f);
    known.store(fn, std::memory_order_release);
  }
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides,
                        boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ADAMAS_OK : cuda_fail(cudaErrorInvalidValue);
}

// The rows of K or V, `box` of them a copy.
static int rows_map(const void* base, int64_t rows, int box, CUtensorMap* map) {
  const cuuint64_t dims[2] = {(cuuint64_t)kDim, (cuuint64_t)rows}, strides[1] = {2 * kDim};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box};
  return tile_map(base, 2, dims, strides, boxes, map);
}

// The queries (or the outputs) [T][Hq][128] for copies of 64 columns, G heads and TQ tokens.
static int query_map(const void* q, int T, int Hq, int G, int TQ, CUtensorMap* map) {
  const cuuint64_t dims[3] = {(cuuint64_t)kDim, (cuuint64_t)Hq, (cuuint64_t)T};
  const cuuint64_t strides[2] = {2 * kDim, (cuuint64_t)Hq * 2 * kDim};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)G, (cuuint32_t)TQ};
  return tile_map(q, 3, dims, strides, boxes, map);
}

// Rows of one tensor-map copy of a 128-row tile: all of them, or the largest power of two
// that divides the page size, of at least 8 rows (the swizzle's period); else 0.
static int rows_box(const CacheGeom& g, int page_size) {
  int box = 128;
  if (g.table)
    while (box >= 8 && page_size % box != 0) box >>= 1;
  return box >= 8 ? box : 0;
}

static int64_t cache_rows(const adamas_chunk_args& a, const CacheGeom& g) {
  return a.block_table ? a.n_pages * a.Hkv * a.page_size : (int64_t)a.B * a.Hkv * g.Nmax;
}

// Workspace of chunk attention: control words | arrival counters | partial states.
static int part_rows(int T, int G) {
  const int tu = 2 * (128 / G);
  return (T < tu ? T : tu) * G;
}
constexpr size_t kAtArrivedBytes = 1024;
static_assert(kAtMaxGrid * sizeof(uint32_t) <= kAtArrivedBytes, "a counter per block");

static int fill_chunk(const adamas_chunk_args& a, bool attend, ChunkParams* p) {
  int rc = check_heads(a.B, a.Hq, a.Hkv, a.d);
  if (rc != ADAMAS_OK) return rc;
  if (a.T < 0) return ADAMAS_ERR_INVALID_ARG;
  if ((rc = make_geom(a.block_table, a.n_pages, a.page_size, a.max_pages, a.Nmax, a.Hkv, &p->geo)) != ADAMAS_OK)
    return rc;
  if (a.B == 0 || a.T == 0) return ADAMAS_OK;
  if (!a.q || !a.cu_q || !a.seq_lens || (p->geo.Nmax > 0 && (!a.K || (attend && !a.V)))) return ADAMAS_ERR_INVALID_ARG;
  if (attend ? !a.out : (!a.lse || (p->geo.Nmax > 0 && !a.mass))) return ADAMAS_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.K, 16) || !aligned(a.V, 16) || !aligned(a.out, 16) || !aligned(a.lse, 4) ||
      !aligned(a.mass, 4) || !aligned(a.cu_q, 4) || !aligned(a.seq_lens, 4))
    return ADAMAS_ERR_INVALID_ARG;
  p->q = static_cast<const uint16_t*>(a.q);
  p->K = static_cast<const uint16_t*>(a.K);
  p->V = static_cast<const uint16_t*>(a.V);
  p->cu_q = a.cu_q;
  p->seq_lens = a.seq_lens;
  p->T = a.T;
  p->B = a.B;
  p->Hq = a.Hq;
  p->Hkv = a.Hkv;
  p->G = a.Hq / a.Hkv;
  p->out = static_cast<uint16_t*>(a.out);
  p->lse = a.lse;
  p->mass = a.mass;
  return ADAMAS_OK;
}

}  // namespace adamas

using namespace adamas;

extern "C" {

int adamas_rope_append(const adamas_rope_args* args, adamas_stream_t stream) {
  if (!args) return ADAMAS_ERR_INVALID_ARG;
  const adamas_rope_args& a = *args;
  int rc = check_heads(a.B, a.Hq, a.Hkv, a.d);
  if (rc != ADAMAS_OK) return rc;
  if (a.T < 0 || a.rot_dim < 0 || a.rot_dim > kDim || a.rot_dim % 2 != 0) return ADAMAS_ERR_INVALID_ARG;
  RopeParams p = {};
  if ((rc = make_geom(a.block_table, a.n_pages, a.page_size, a.max_pages, a.Nmax, a.Hkv, &p.geo)) != ADAMAS_OK)
    return rc;
  if ((a.k == nullptr) != (a.v == nullptr)) return ADAMAS_ERR_INVALID_ARG;
  if (a.B == 0 || a.T == 0 || (!a.q && !a.k)) return ADAMAS_OK;
  if (!a.cu_new || !a.cache_lens || (a.rot_dim > 0 && !a.freqs)) return ADAMAS_ERR_INVALID_ARG;
  if (a.q && (!a.q_out || !aligned(a.q, 16) || !aligned(a.q_out, 16) || a.q_stride < (int64_t)a.Hq * kDim ||
              a.q_stride % 8 != 0 || (a.q_out == a.q && a.q_stride != (int64_t)a.Hq * kDim)))
    return ADAMAS_ERR_INVALID_ARG;
  if (a.k && ((p.geo.Nmax > 0 && (!a.K || !a.V)) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.K, 16) ||
              !aligned(a.V, 16) || !aligned(a.codes, 32) || a.k_stride < (int64_t)a.Hkv * kDim ||
              a.v_stride < (int64_t)a.Hkv * kDim || a.k_stride % 8 != 0 || a.v_stride % 8 != 0))
    return ADAMAS_ERR_INVALID_ARG;
  if (!aligned(a.cu_new, 4) || !aligned(a.cache_lens, 4) || !aligned(a.positions, 4) || !aligned(a.freqs, 8))
    return ADAMAS_ERR_INVALID_ARG;
  if ((rc = check_ctrl(a.workspace, a.workspace_bytes, kCtrlBytes)) != ADAMAS_OK) return rc;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.cu_new = a.cu_new;
  p.cache_lens = a.cache_lens;
  p.positions = a.positions;
  p.freqs = a.freqs;
  p.rot = a.rot_dim;
  p.mscale = a.mscale;
  p.T = a.T;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.K = static_cast<uint16_t*>(a.K);
  p.V = static_cast<uint16_t*>(a.V);
  p.codes = a.codes;
  p.err = err_word(a.workspace);
  // many tokens: kRopeTokens to a block; a few: one, and its rows over more blocks, down to
  // two rows a warp, as the rows of a warp come one after the other
  const int pairs = ((p.q ? a.Hq : 0) + (p.k ? 2 * a.Hkv : 0) + 1) / 2, warps = kRopeThreads / 32;
  int split = (pairs + warps - 1) / warps;
  if ((int64_t)split * a.T > kRopeSplitBlocks) split = (int)(kRopeSplitBlocks / a.T > 0 ? kRopeSplitBlocks / a.T : 1);
  p.neg0 = 0x8000000080000000ull;
  p.tokens = a.T >= kRopeSplitBlocks * kRopeTokens ? kRopeTokens : 1;
  const dim3 grid((unsigned)((a.T + p.tokens - 1) / p.tokens), (unsigned)split);
  cudaStream_t st = (cudaStream_t)stream;
  if (a.interleaved) rope_append_kernel<kRopeInside><<<grid, kRopeThreads, 0, st>>>(p);
  else if (a.rot_dim % 16 == 0) rope_append_kernel<kRopeShuffle><<<grid, kRopeThreads, 0, st>>>(p);
  else rope_append_kernel<kRopeLoad><<<grid, kRopeThreads, 0, st>>>(p);
  return launched();
}

size_t adamas_chunk_workspace_bytes(int T, int B, int Hq, int Hkv, int d) {
  if (T < 0 || check_heads(B, Hq, Hkv, d) != ADAMAS_OK) return 0;
  return kCtrlBytes + kAtArrivedBytes + (size_t)2 * kAtMaxGrid * part_rows(T, Hq / Hkv) * kAtPartRow * sizeof(float);
}

int adamas_chunk_attend(const adamas_chunk_args* args, adamas_stream_t stream) {
  if (!args) return ADAMAS_ERR_INVALID_ARG;
  const adamas_chunk_args& a = *args;
  ChunkParams p = {};
  int rc = fill_chunk(a, true, &p);
  if (rc != ADAMAS_OK || a.B == 0 || a.T == 0) return rc;
  if ((rc = check_ctrl(a.workspace, a.workspace_bytes, adamas_chunk_workspace_bytes(a.T, a.B, a.Hq, a.Hkv, a.d))) !=
      ADAMAS_OK)
    return rc;
  p.err = err_word(a.workspace);
  int sms = 0;
  if ((rc = attend_device(&sms)) != ADAMAS_OK) return rc;
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  AtParams ap;
  ap.c = p;
  ap.arrived = reinterpret_cast<uint32_t*>(ws + kCtrlBytes);
  ap.part = reinterpret_cast<float*>(ws + kCtrlBytes + kAtArrivedBytes);
  ap.part_rows = part_rows(a.T, p.G);
  ap.TQ = 128 / p.G;
  const int64_t rows = cache_rows(a, p.geo);
  if (rows > INT32_MAX) return ADAMAS_ERR_UNSUPPORTED;
  CUtensorMap q_map = {}, k_map = {}, v_map = {}, o_map = {};
  if ((rc = query_map(a.q, a.T, a.Hq, p.G, ap.TQ, &q_map)) != ADAMAS_OK) return rc;
  ap.out_copies = 32 % p.G == 0;
  if (ap.out_copies && (rc = query_map(a.out, a.T, a.Hq, p.G, 32 / p.G, &o_map)) != ADAMAS_OK) return rc;
  ap.box = rows > 0 ? rows_box(p.geo, a.page_size) : 0;
  if (ap.box && ((rc = rows_map(a.K, rows, ap.box, &k_map)) != ADAMAS_OK ||
                 (rc = rows_map(a.V, rows, ap.box, &v_map)) != ADAMAS_OK))
    return rc;
  // no more blocks than K/V tiles of all units
  const int64_t units = (int64_t)p.Hkv * ((a.T + 2 * ap.TQ - 1) / (2 * ap.TQ) + p.B);
  const int64_t tiles = units * ((p.geo.Nmax + 127) / 128 + 1);
  chunk_attend_kernel<<<(unsigned)(tiles < sms ? tiles : sms), kAtThreads, kAtSmem, (cudaStream_t)stream>>>(
      ap, q_map, k_map, v_map, o_map);
  return launched();
}

int adamas_accumulate_chunk(const adamas_chunk_args* args, adamas_stream_t stream) {
  if (!args) return ADAMAS_ERR_INVALID_ARG;
  const adamas_chunk_args& a = *args;
  ChunkParams p = {};
  int rc = fill_chunk(a, false, &p);
  if (rc != ADAMAS_OK || a.B == 0 || a.T == 0 || p.geo.Nmax == 0) return rc;
  if ((rc = check_ctrl(a.workspace, a.workspace_bytes, kCtrlBytes)) != ADAMAS_OK) return rc;
  p.err = err_word(a.workspace);
  int sms = 0;
  if ((rc = attend_device(&sms)) != ADAMAS_OK) return rc;
  const int64_t rows = cache_rows(a, p.geo);
  const int64_t units = (int64_t)a.B * a.Hkv * ((p.geo.Nmax + 255) / 256);
  if (rows > INT32_MAX || units > INT32_MAX) return ADAMAS_ERR_UNSUPPORTED;
  WtParams wp;
  wp.c = p;
  wp.TQ = 128 / p.G;
  wp.box = rows_box(p.geo, a.page_size);
  CUtensorMap q_map = {}, k_map = {};
  if ((rc = query_map(a.q, a.T, a.Hq, p.G, wp.TQ, &q_map)) != ADAMAS_OK) return rc;
  if (wp.box && (rc = rows_map(a.K, rows, wp.box, &k_map)) != ADAMAS_OK) return rc;
  chunk_weights_kernel<<<(unsigned)(units < sms ? units : sms), kWtThreads, kWtSmem, (cudaStream_t)stream>>>(wp, q_map,
                                                                                                             k_map);
  return launched();
}

int adamas_accumulate_kept(const adamas_kept_args* args, adamas_stream_t stream) {
  if (!args) return ADAMAS_ERR_INVALID_ARG;
  const adamas_kept_args& a = *args;
  int rc = check_heads(a.B, a.Hq, a.Hkv, a.d);
  if (rc != ADAMAS_OK) return rc;
  if (a.budget < 0 || (a.policy != ADAMAS_SELECT_PER_HEAD && a.policy != ADAMAS_SELECT_GROUP_SHARED))
    return ADAMAS_ERR_INVALID_ARG;
  KeptParams p = {};
  if ((rc = make_geom(a.block_table, a.n_pages, a.page_size, a.max_pages, a.Nmax, a.Hkv, &p.geo)) != ADAMAS_OK)
    return rc;
  if (a.B == 0 || a.budget == 0 || p.geo.Nmax == 0) return ADAMAS_OK;
  if (!a.q || !a.K || !a.idx || !a.seq_lens || !a.mass) return ADAMAS_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.K, 16) || !aligned(a.idx, 4) || !aligned(a.seq_lens, 4) || !aligned(a.mass, 4))
    return ADAMAS_ERR_INVALID_ARG;
  if ((rc = check_ctrl(a.workspace, a.workspace_bytes, kCtrlBytes)) != ADAMAS_OK) return rc;
  p.q = static_cast<const uint16_t*>(a.q);
  p.K = static_cast<const uint16_t*>(a.K);
  p.idx = a.idx;
  p.seq_lens = a.seq_lens;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.budget = a.budget;
  p.shared_rows = a.policy == ADAMAS_SELECT_GROUP_SHARED;
  p.mass = a.mass;
  p.err = err_word(a.workspace);
  // blocks of a kv head: up to about two per multiprocessor in all, 64 slots of a list each
  // at least; more when a block's scores would not fit
  const int heads = a.B * a.Hkv;
  int C = 1;
  while (C < kKeptCluster && (int64_t)heads * 2 * C <= 296 && a.budget >= 128 * C) C *= 2;
  while (C < kKeptCluster && (int64_t)((a.budget + C - 1) / C) * p.G > kKeptSmemFloats) C *= 2;
  const int cap = (a.budget + C - 1) / C;
  if ((int64_t)cap * p.G > kKeptSmemFloats) {
    accumulate_kept_large_kernel<<<(unsigned)heads, 256, 0, (cudaStream_t)stream>>>(p);
    return launched();
  }
  return launch_cluster<accumulate_kept_kernel>(heads * C, C, kKeptThreads, (size_t)cap * p.G * sizeof(float),
                        kKeptSmemFloats * sizeof(float), false, (cudaStream_t)stream, p, cap);
}

int adamas_evict(const adamas_evict_args* args, adamas_stream_t stream) {
  if (!args) return ADAMAS_ERR_INVALID_ARG;
  const adamas_evict_args& a = *args;
  int rc = check_heads(a.B, a.Hkv, a.Hkv, a.d);
  if (rc != ADAMAS_OK) return rc;
  if (a.keep < 0 || a.n_sink < 0 || a.n_recent < 0) return ADAMAS_ERR_INVALID_ARG;
  EvictParams p = {};
  if ((rc = make_geom(a.block_table, a.n_pages, a.page_size, a.max_pages, a.Nmax, a.Hkv, &p.geo)) != ADAMAS_OK)
    return rc;
  const bool in_place = !a.K_out && !a.V_out && !a.codes_out && !a.mass_out && !a.block_table_out;
  if (in_place) {
    p.out = p.geo;
  } else {
    if ((rc = make_geom(a.block_table_out, a.n_pages_out, a.page_size_out, a.max_pages_out, a.Nmax_out, a.Hkv,
                        &p.out)) != ADAMAS_OK)
      return rc;
    if (p.out.Nmax < a.keep) return ADAMAS_ERR_INVALID_ARG;
    if ((a.codes == nullptr) != (a.codes_out == nullptr)) return ADAMAS_ERR_INVALID_ARG;
  }
  if (a.B == 0 || (p.geo.Nmax == 0 && p.out.Nmax == 0)) return ADAMAS_OK;
  if (!a.seq_lens || !a.new_lens || a.new_lens == a.seq_lens || (a.keep > 0 && !a.kept)) return ADAMAS_ERR_INVALID_ARG;
  if (p.geo.Nmax > 0 && (!a.K || !a.V || !a.mass)) return ADAMAS_ERR_INVALID_ARG;
  if (!in_place && ((a.keep > 0 && (!a.K_out || !a.V_out)) || !a.mass_out || a.K_out == a.K || a.V_out == a.V ||
                    a.mass_out == a.mass || (a.codes && a.codes_out == a.codes)))
    return ADAMAS_ERR_INVALID_ARG;
  if (!aligned(a.K, 16) || !aligned(a.V, 16) || !aligned(a.codes, 32) || !aligned(a.mass, 4) || !aligned(a.K_out, 16) ||
      !aligned(a.V_out, 16) || !aligned(a.codes_out, 32) || !aligned(a.mass_out, 4) || !aligned(a.kept, 4) ||
      !aligned(a.seq_lens, 4) || !aligned(a.new_lens, 4))
    return ADAMAS_ERR_INVALID_ARG;
  if ((rc = check_ctrl(a.workspace, a.workspace_bytes, kCtrlBytes)) != ADAMAS_OK) return rc;
  p.K = static_cast<const uint16_t*>(a.K);
  p.V = static_cast<const uint16_t*>(a.V);
  p.codes = a.codes;
  p.mass = a.mass;
  p.seq_lens = a.seq_lens;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.keep = a.keep;
  p.n_sink = a.n_sink;
  p.n_recent = a.n_recent;
  p.kept = a.kept;
  p.new_lens = a.new_lens;
  p.K_out = static_cast<uint16_t*>(in_place ? a.K : a.K_out);
  p.V_out = static_cast<uint16_t*>(in_place ? a.V : a.V_out);
  p.codes_out = in_place ? a.codes : a.codes_out;
  p.mass_out = in_place ? a.mass : a.mass_out;
  p.err = err_word(a.workspace);
  cudaStream_t st = (cudaStream_t)stream;
  const int heads = a.B * a.Hkv;
  int C = (int)((p.geo.Nmax + kSelBlockTokens - 1) / kSelBlockTokens);
  C = C < 1 ? 1 : (C > kSelCluster ? kSelCluster : C);
  const int64_t slice = (p.geo.Nmax + C - 1) / C;
  p.smem_keys = slice <= kSelSmemTokens ? (int)slice : kSelSmemSome;
  if ((rc = launch_cluster<evict_select_kernel>(heads * C, C, kSelThreads, (size_t)p.smem_keys * sizeof(uint32_t),
                                                kSelSmemTokens * sizeof(uint32_t), false, st, p)) != ADAMAS_OK)
    return rc;
  if (in_place) {  // a cluster per head, up to about one block per multiprocessor in all
    C = 1;
    while (C < 8 && (int64_t)heads * 2 * C <= 148 && a.keep >= 64 * C) C *= 2;
    return launch_cluster<evict_shift_kernel>(heads * C, C, kShiftThreads, 0, 0, true, st, p);
  }
  int per_head = (int)(((int64_t)a.keep + 31) / 32);  // a round of a block's warps at least
  const int most = kCopyBlocks / heads;
  if (per_head > most) per_head = most;
  if (per_head < 1) per_head = 1;
  return launch_cluster<evict_copy_kernel>(heads * per_head, 1, kMoveThreads, 0, 0, true, st, p, per_head);
}

}  // extern "C"
