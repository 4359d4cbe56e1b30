/*
 * adamas.h -- C ABI of the B200 (sm_100a) ADAMAS sparse decode attention library.
 *
 * The method is the one described in the ADAMAS long-context sparse attention
 * article (lnwmold.com/news/826806):
 *   §2.1  queries and cached keys are rotated by an orthogonal Hadamard matrix,
 *         which leaves every q.k unchanged and spreads outlier channels;
 *   §2.2  each rotated vector is bucketed into 2-bit codes by three dynamic
 *         thresholds (-m/2, 0, +m/2), m = max |y| over the 128-dim group;
 *   §3.1  the codes are kept as a packed cache, four codes per byte;
 *   §2.3  every cached token is scored by the Manhattan (L1) distance between
 *         its codes and the query's codes (a smaller distance is more relevant);
 *   §5.2  only a token budget of the best-scoring tokens is kept, and exact
 *         softmax attention runs over the K/V rows of those tokens.
 *
 * Conventions shared by every entry point
 *   - Head dimension d must be 128 (one bucketing group per vector).
 *   - Tensors are dense row-major in device memory:
 *       q       [B][Hq][128]          bf16
 *       K, V    [B][Hkv][Nmax][128]   bf16
 *       codes   [B][Hkv][Nmax][32]    uint8, four 2-bit codes per byte, the code of
 *                                     dimension 4j in bits 7:6 of byte j
 *       out     [B][Hq][128]          fp32
 *       idx     [B][Hq][budget]       int32
 *     Query head h reads kv head h / (Hq / Hkv) (grouped-query attention).
 *   - The caller owns every buffer and the stream.  Calls only enqueue work on
 *     `stream` (a cudaStream_t; NULL is the legacy default stream) and return;
 *     they never allocate, free or synchronise, except adamas_get_device_error,
 *     which synchronises `stream` to read the error word.
 *   - codes must be 32-byte aligned (it is streamed with 32-byte loads); the
 *     other bf16/fp32 tensors and the workspace 16-byte aligned; int32 arrays
 *     4-byte aligned.  Inputs must be finite: NaN or Inf in q or K gives
 *     unspecified codes, indices and outputs (never an out-of-bounds access).
 *   - Argument errors are detected on the host before anything is enqueued and
 *     are returned as a negative status; nothing is written in that case.  A
 *     failed launch returns ADAMAS_ERR_CUDA.  Conditions only the GPU can see
 *     (a sequence length outside [0, Nmax], a cross-block wait that timed out)
 *     set bits of an error word in the workspace; see adamas_get_device_error.
 *   - No exception crosses this interface.  All entry points are thread-safe
 *     for distinct workspaces.
 */
#ifndef ADAMAS_H
#define ADAMAS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without including the CUDA runtime headers */
typedef struct CUstream_st *adamas_stream_t;

enum adamas_status {
    ADAMAS_OK = 0,
    ADAMAS_ERR_INVALID_ARG = -1, /* null/misaligned pointer, bad size or shape */
    ADAMAS_ERR_UNSUPPORTED = -2, /* d != 128, group size > 8, batch > 1024, ... */
    ADAMAS_ERR_WORKSPACE = -3,   /* workspace missing or smaller than adamas_workspace_bytes */
    ADAMAS_ERR_CUDA = -4,        /* a CUDA runtime call or kernel launch failed */
    ADAMAS_ERR_DEVICE = -5       /* the device error word is non-zero */
};

/* Bits of the device error word. */
#define ADAMAS_DEVERR_SEQLEN 0x1u  /* a seq_lens entry was outside [0, Nmax]; it was clamped */
#define ADAMAS_DEVERR_TIMEOUT 0x2u /* a bounded wait on a stage copy gave up; the step's outputs are invalid */
#define ADAMAS_DEVERR_INTERNAL 0x4u /* a block's share exceeded its planned size; outputs are invalid */
#define ADAMAS_DEVERR_TABLE 0x8u    /* a block-table entry was outside [0, n_pages); page 0 was read instead
                                       (calls that write through the table write nothing there) */
#define ADAMAS_DEVERR_OFFSETS 0x10u /* offsets of a ragged batch were not ascending within [0, T] */

/* Selection policies of adamas_decode_step_ex. */
enum adamas_select_policy {
    ADAMAS_SELECT_PER_HEAD = 0,    /* every query head keeps its own budget of tokens */
    ADAMAS_SELECT_GROUP_SHARED = 1 /* one budget per kv head, ranked by the distance summed over its query heads */
};

/* Static description of a status code (never NULL). */
const char *adamas_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int adamas_version(void);

/* Text of the last CUDA error that made a call of this thread return
 * ADAMAS_ERR_CUDA ("no CUDA error" if none).  Never NULL. */
const char *adamas_last_error_string(void);

/*
 * Bytes of device workspace adamas_decode_step needs for these sizes on the
 * current CUDA device (0 when the sizes are unsupported).  The workspace holds
 * the device error word and, only when a block's token distances do not fit in
 * shared memory (very long contexts), a spill area for them; histograms and
 * partial softmax states stay on chip.  For long contexts over few kv heads
 * (fewer clusters than fill 3/4 of the SMs, at least 65,536 tokens) the step
 * splits every (b, kv head) into slices inside the GPU, and the workspace also
 * carries the slices' histograms and softmax states.  It must be zero-filled once
 * before its first use (adamas_workspace_init); every step leaves it ready for the
 * next one.  One workspace must not be used by two steps that may run
 * concurrently.
 */
size_t adamas_workspace_bytes(int B, int Hq, int Hkv, int64_t Nmax, int d, int budget);

/* Zero-fill a workspace on `stream` (asynchronous).  Also the way to clear the
 * error word and recover after ADAMAS_DEVERR_TIMEOUT. */
int adamas_workspace_init(void *workspace, size_t workspace_bytes, adamas_stream_t stream);

/*
 * Encode cached keys into packed 2-bit codes (article §2.1 rotation, §2.2
 * bucketing, §3.1 packing).  For every (b, kv head) it encodes positions
 * [p, p + count) with p = pos_begin[b] (pos_begin: device int32[B], or NULL for
 * p = 0); positions outside [0, Nmax) are skipped.  Use count = Nmax at prefill
 * and count = 1 with pos_begin = the new token's position when appending.
 *   K      device bf16 [B][Hkv][Nmax][128]  (read)
 *   codes  device uint8 [B][Hkv][Nmax][32]  (written at the encoded positions)
 * The rotation is an fp32 Sylvester-order butterfly (stage widths 1..64, no
 * fused multiply-add) followed by one multiply by RN(1/sqrt(128)); the codes are
 * bit-identical to the CPU oracle's.
 */
int adamas_encode_keys(const void *K, uint8_t *codes, const int32_t *pos_begin, int count, int B,
                       int Hkv, int64_t Nmax, int d, adamas_stream_t stream);

/*
 * One decode step of one attention layer for the whole batch: encode q, score
 * every cached token t < seq_lens[b] of the query head's kv head by the L1
 * distance D of the codes (article §2.3), keep k_eff = min(budget, seq_lens[b])
 * tokens of smallest (D, t) -- ties go to the lower token index -- and run exact
 * softmax attention with scale 1/sqrt(128) over their bf16 K/V rows, in fp32.
 *   q         device bf16 [B][Hq][128]
 *   codes     device uint8 [B][Hkv][Nmax][32]  (from adamas_encode_keys)
 *   K, V      device bf16 [B][Hkv][Nmax][128]
 *   seq_lens  device int32 [B]
 *   out       device fp32 [B][Hq][128]   softmax-weighted sum of the kept V rows
 *                                        (0 when k_eff = 0)
 *   idx       device int32 [B][Hq][budget]  kept token positions in (D, t)
 *                                        order, -1 past k_eff
 *   workspace device, >= adamas_workspace_bytes(...) bytes, zero-filled once
 * The step runs as one kernel launch: one thread-block cluster per (b, kv head),
 * its blocks splitting the head's tokens and exchanging histograms and partial
 * softmax states through distributed shared memory.  The launch opts in to
 * programmatic dependent launch: its blocks may be scheduled while the previous
 * kernel of the stream drains, and each waits for that kernel to complete (and
 * its writes to be visible) before its first global read or write, so stream
 * order semantics are unchanged.
 */
int adamas_decode_step(const void *q, const uint8_t *codes, const void *K, const void *V,
                       const int32_t *seq_lens, int B, int Hq, int Hkv, int64_t Nmax, int d,
                       int budget, float *out, int32_t *idx, void *workspace,
                       size_t workspace_bytes, adamas_stream_t stream);

/*
 * adamas_encode_keys for one appended token per sequence followed by
 * adamas_decode_step, in one launch -- the usual decode-loop step (article §3.1:
 * the code cache grows by one row per generated token; §2.3, §5.2: the step then
 * scores and selects over the whole cache).  For every (b, kv head) with
 * 0 <= append_pos[b] < Nmax, the key K[b][kvh][append_pos[b]] (already written by
 * the caller) is encoded into codes exactly as adamas_encode_keys would, before
 * the step scores that position; other values of append_pos[b] append nothing.
 *   codes       device uint8 [B][Hkv][Nmax][32], read and written
 *   append_pos  device int32 [B]
 * Every other argument, result and rule is adamas_decode_step's; the results are
 * bit-identical to adamas_encode_keys(count 1, pos_begin = append_pos) followed
 * by adamas_decode_step.
 */
int adamas_decode_step_append(const void *q, uint8_t *codes, const void *K, const void *V,
                              const int32_t *seq_lens, const int32_t *append_pos, int B, int Hq,
                              int Hkv, int64_t Nmax, int d, int budget, float *out, int32_t *idx,
                              void *workspace, size_t workspace_bytes, adamas_stream_t stream);

/*
 * Debug and test entry point: the distances the decode step ranks by.
 *   dist  device uint16 [B][Hq][Nmax]: D in [0, 384] for t < seq_lens[b],
 *         0xFFFF past the sequence length.
 * Same argument rules as adamas_decode_step; seq_lens outside [0, Nmax] are
 * clamped (no error word here).
 */
int adamas_score(const void *q, const uint8_t *codes, const int32_t *seq_lens, int B, int Hq,
                 int Hkv, int64_t Nmax, int d, uint16_t *dist, adamas_stream_t stream);

/*
 * adamas_decode_step for callers that cannot allocate device memory where they
 * decode -- an allocator that must not be re-entered from the decode loop, a hook
 * that runs with allocation forbidden, or a program that only receives pointers
 * to memory someone else owns.  The ADAMAS article has no counterpart of this
 * entry point; it is a property of this library.
 *
 * Same arguments, results and rules as adamas_decode_step, without the
 * workspace: the scratch is a fixed 4 MiB array that the library keeps in the
 * global memory of every device it is loaded on, until the process exits.
 * Nothing is allocated or freed by this call.
 *   - Sizes whose workspace (adamas_workspace_bytes) exceeds 4 MiB are rejected
 *     with ADAMAS_ERR_WORKSPACE before anything is enqueued; use
 *     adamas_decode_step for those.
 *   - Every call on a device shares the one array, and it keeps the previous
 *     call's contents.  The call clears what must start at zero, but calls that
 *     may overlap on the GPU (different streams, or different threads without
 *     ordering) race on it; serialise them.
 *   - The device error word lives in the shared array; every call clears it
 *     first.  adamas_static_device_error reads the last call's word.
 *   - The array's address is looked up once per CUDA context (keyed by the
 *     context's process-unique id) and cached.  cudaDeviceReset destroys the
 *     context and the array's contents with it; the next call, in the new
 *     context, looks the address up again.
 */
int adamas_decode_step_static(const void *q, const uint8_t *codes, const void *K, const void *V,
                              const int32_t *seq_lens, int B, int Hq, int Hkv, int64_t Nmax, int d,
                              int budget, float *out, int32_t *idx, adamas_stream_t stream);

/*
 * Reads the device error word of the last adamas_decode_step_static call on the
 * current device (the word lives in the fixed scratch array; see
 * adamas_get_device_error for its bits).  Synchronises `stream`, so call it on
 * the stream of the decode calls, after them.  The word stays until the next
 * static call clears it.
 * Returns ADAMAS_OK when the word is 0, ADAMAS_ERR_DEVICE when a bit is set
 * (*error_word holds them), ADAMAS_ERR_INVALID_ARG for a NULL error_word,
 * ADAMAS_ERR_CUDA when the copy fails.
 */
int adamas_static_device_error(uint32_t *error_word, adamas_stream_t stream);

/*
 * Every option of the decode step in one call.  adamas_decode_step and
 * adamas_decode_step_append are this call with the optional fields zero.
 *
 * Required fields (as in adamas_decode_step):
 *   q, codes, K, V, seq_lens, B, Hq, Hkv, Nmax, d, budget, out, idx,
 *   workspace, workspace_bytes
 *
 * Optional fields (zero / NULL: off):
 *   append_pos   device int32 [B]: the key at append_pos[b] is encoded into codes
 *                before the step scores it (adamas_decode_step_append; the ADAMAS
 *                article's §3.1: the code cache grows by one row per token).
 *   k_new, v_new device bf16 [B][Hkv][128], both or neither, only with append_pos:
 *                the launch itself writes these rows into K and V at append_pos[b]
 *                (and encodes k_new), so a decode loop needs no separate copy of the
 *                new token's rows into the cache.  K and V are written.
 *   block_table  device int32 [B][max_pages]: a paged cache.  Token t of sequence b
 *                lives in physical page block_table[b][t / page_size] at slot
 *                t % page_size; codes, K and V are then page arrays laid out
 *                [n_pages][Hkv][page_size][32 or 128] (every kv head's rows of a page
 *                contiguous), and Nmax is ignored (max_pages * page_size tokens per
 *                sequence).  adamas_encode_keys encodes such a cache as B = n_pages
 *                sequences of Nmax = page_size tokens.  An entry outside
 *                [0, n_pages) sets ADAMAS_DEVERR_TABLE (the step then reads page 0).
 *                Requires n_pages * Hkv * page_size <= 2^31 - 1.
 *   page_size, max_pages, n_pages   the paged cache's geometry.
 *   n_sink, n_recent  forced rows: the first n_sink and the last n_recent tokens of
 *                every sequence rank ahead of every scored token (in index order), as
 *                attention sinks and a recent window; the rest are ranked by (D, t).
 *                When they outnumber k_eff the lowest indices win.
 *   policy       ADAMAS_SELECT_PER_HEAD (default) or ADAMAS_SELECT_GROUP_SHARED: for
 *                every (b, kv head) the distances of its G query heads are summed per
 *                token, k_eff tokens of smallest (sum, t) are kept once, and every
 *                query head of the group attends over them; idx is then
 *                [B][Hkv][budget] and budget must be <= 4096 (ADAMAS_ERR_UNSUPPORTED
 *                otherwise).  The K/V rows are read once per kv head instead of once
 *                per query head.
 * The grouped-head and forced-row rules are readings of the article's §2.3 and
 * §5.2 (which state the scoring and the budget per head) and of its §3.2 and §6
 * tuning advice (some tokens keep full attention); the paged layout follows the
 * block-table caches that paged-attention serving uses.  Same errors and
 * asynchrony as adamas_decode_step; the workspace size is adamas_workspace_bytes of
 * (B, Hq, Hkv, Nmax, d, budget) with Nmax = max_pages * page_size when paged.
 */
typedef struct adamas_decode_args {
    const void *q;
    uint8_t *codes;
    void *K;
    void *V;
    const int32_t *seq_lens;
    int B, Hq, Hkv;
    int64_t Nmax;
    int d;
    int budget;
    float *out;
    int32_t *idx;
    void *workspace;
    size_t workspace_bytes;
    const int32_t *append_pos;
    const void *k_new;
    const void *v_new;
    const int32_t *block_table;
    int64_t n_pages;
    int page_size;
    int max_pages;
    int n_sink;
    int n_recent;
    int policy;
} adamas_decode_args;

int adamas_decode_step_ex(const adamas_decode_args *args, adamas_stream_t stream);

/*
 * Test hook (not for production use): from now on every decode step runs its
 * general kernel and never issues the bulk copy of code stage `stage` in any
 * block, so the workers' bounded wait for that stage gives up after about a
 * second, sets ADAMAS_DEVERR_TIMEOUT and the step completes with invalid outputs;
 * no copy is left in flight.  A negative `stage` turns the hook off.  Process-wide
 * and not thread-safe: for the tests of the timeout path only.
 */
void adamas_debug_withhold_stage(int stage);

/*
 * Sequence-sharded decode step, for contexts longer than one GPU holds (the 2M-token
 * context blog, intelliparadigm.com/.../2174157, §5.1: two million tokens need
 * several GPUs or CPU offloading; the AMD Zebra-HyLo article,
 * yeyulingfeng.com/a/1106654.html, reports 2M-token contexts).  Each of `world`
 * GPUs holds one contiguous slice of every sequence (rank r the r-th slice, in
 * sequence order) in its own codes/K/V arrays, [B][Hkv][Nmax][...] as above with
 * seq_lens[b] the slice's length.  One step, on every rank:
 *   1. adamas_shard_score: scores the slice; writes the slice's distance
 *      histograms to `hist` [B][Hq][ADAMAS_HIST_STRIDE] uint32 (bins 0..384).
 *   2. all-gather of `hist` in rank order -> hist_all [world][B][Hq][ADAMAS_HIST_STRIDE].
 *   3. adamas_shard_attend: from hist_all, the threshold and rank bases of the
 *      whole sequence (k_eff = min(budget, total length)); the slice's kept tokens
 *      get their slots, idx [B][Hq][budget] holds their indices in the whole
 *      sequence (every other slot -1), and `partial` [B][Hq][ADAMAS_PARTIAL_FLOATS]
 *      fp32 receives the slice's softmax state over them.
 *   4. all-gather of `partial` -> [world][B][Hq][ADAMAS_PARTIAL_FLOATS], and an
 *      all-reduce (max) of idx.
 *   5. adamas_merge_partials -> out [B][Hq][128].
 * The result is the step of adamas_decode_step on the whole sequence: the same
 * idx, and out within the float tolerance of the single-GPU step.  Per head and
 * rank the messages are 388 * 4 B (histograms) and 132 * 4 B (state) plus the idx
 * row.  Per-head selection only (no forced rows, paged cache, group-shared policy
 * or append); global indices are int32, so a sequence holds at most 2^31 - 1 tokens.
 *
 * The workspace (adamas_shard_workspace_bytes, initialised once with
 * adamas_workspace_init) carries the slice's distances and per-block histograms
 * from step 1 to step 3: use the same workspace, stream and shape for both.
 * `hist` and idx are overwritten (zeroed / set to -1) by the calls themselves.
 * A partial state is (m, l, 0, 0, o[128]): m the largest score of the slice's kept
 * tokens, in log2 units (q.k / sqrt(128) * log2 e), l = sum 2^(s - m) and
 * o = sum 2^(s - m) v over them; m = -inf and l = 0 when the slice kept none.
 * Errors as for adamas_decode_step; the device error word is the workspace's.
 */
#define ADAMAS_HIST_STRIDE 388
#define ADAMAS_PARTIAL_FLOATS 132

size_t adamas_shard_workspace_bytes(int B, int Hq, int Hkv, int64_t Nmax, int d, int budget);

int adamas_shard_score(const void *q, const uint8_t *codes, const int32_t *seq_lens, int B, int Hq, int Hkv,
                       int64_t Nmax, int d, int budget, uint32_t *hist, void *workspace, size_t workspace_bytes,
                       adamas_stream_t stream);

/* world >= 1 ranks, 0 <= rank < world; hist_all as gathered in step 2. */
int adamas_shard_attend(const void *q, const void *K, const void *V, const int32_t *seq_lens, int B, int Hq, int Hkv,
                        int64_t Nmax, int d, int budget, const uint32_t *hist_all, int world, int rank,
                        float *partial, int32_t *idx, void *workspace, size_t workspace_bytes,
                        adamas_stream_t stream);

/*
 * out[b][h][e] = sum_r 2^(m_r - M) o_r[e] / sum_r 2^(m_r - M) l_r over the n states
 * partials [n][B][Hq][ADAMAS_PARTIAL_FLOATS] (M = max_r m_r; states with m_r = -inf
 * are skipped; 0 when every state is empty).  16-byte aligned fp32 arrays.
 */
int adamas_merge_partials(const float *partials, int n, int B, int Hq, float *out, adamas_stream_t stream);

/* ======================================================================== cache operators
 * What a serving loop runs around the decode step, over the same cache: rotary
 * positions and the append of new rows, attention of a chunk of new tokens, the
 * attention weight that each cached token has received, and the eviction of the
 * tokens that received least.
 *
 * Shared conventions (besides the ones at the top of this file)
 *   - A cache is contiguous, K and V [B][Hkv][Nmax][128], or paged (block_table
 *     given): [n_pages][Hkv][page_size][128] read through block_table
 *     [B][max_pages], with Nmax ignored and max_pages * page_size tokens per
 *     sequence, exactly as in adamas_decode_args.  codes follow with 32 B rows.
 *     Token numbers below ("slots") are positions in the sequence's cache.
 *   - A ragged batch of new tokens is packed: sequence b owns rows
 *     [cu[b], cu[b + 1]) of the T rows, cu device int32 [B + 1], ascending within
 *     [0, T] (else ADAMAS_DEVERR_OFFSETS, and the sequence is left out).  Rows
 *     before cu[0] and from cu[B] on belong to no sequence: their values play no
 *     part and their outputs are left as they were.
 *   - mass device fp32 [B][Hkv][Nmax] (paged: Nmax = max_pages * page_size, by slot
 *     and not by page): the attention weight a token received so far, summed over
 *     query rows and over the query heads of its kv head.
 *   - workspace: adamas_chunk_workspace_bytes for adamas_chunk_attend; for the other
 *     calls any workspace of this library (the device error word in its first 256
 *     bytes is all they use).  Zero-filled once (adamas_workspace_init).
 *   - Slots at or past a sequence's length may hold anything, NaN included; rows
 *     inside it must be finite.
 */

/*
 * Rotary positions of new query and key rows, and the append of the new rows to
 * the cache.  Token i of sequence b (row r = cu_new[b] + i) is rotated by its
 * position p = positions[r] (or its slot when positions is NULL) and goes to slot
 * cache_lens[b] + i; a slot outside [0, Nmax) is not written.
 *   pair j of the rotated part (the first rot_dim dimensions; the rest pass
 *   unchanged): dimensions (j, j + rot_dim / 2), or (2j, 2j + 1) when interleaved;
 *   turn = freqs[j] * p mod 2^64, in 2^-64 turns (so p may be any int32, and the
 *   angle of a far position is as exact as that of a near one);
 *   c = RN32(mscale cos), s = RN32(mscale sin) of that angle, evaluated in 64 bits;
 *   (x1, x2) -> (RN32(x1 c) - RN32(x2 s), RN32(x2 c) + RN32(x1 s)), each rounded to
 *   fp32 and then once to bf16: the same bits on every run and batch shape, so that
 *   the codes made from them are reproducible too.
 * codes (optional) receives the packed codes of the rotated keys, as
 * adamas_encode_keys makes them.
 *   q, k, v    device bf16, row r at q + r * q_stride (elements, a multiple of 8;
 *              Hq or Hkv heads of 128 contiguous), so they may be parts of one
 *              projection's output.  q may be NULL (nothing rotated), k and v both
 *              NULL (nothing appended).
 *   q_out      device bf16 [T][Hq][128]; may be q itself when q_stride = Hq * 128.
 *   freqs      device uint64 [rot_dim / 2]: angle per position of each pair as a
 *              fraction of a turn, times 2^64 (scaling methods change this table and mscale)
 *   rot_dim    even, 0..128
 * The slots written in one call must be distinct.
 */
typedef struct adamas_rope_args {
    const void *q;
    const void *k;
    const void *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu_new;
    const int32_t *cache_lens;
    const int32_t *positions;
    const uint64_t *freqs;
    int rot_dim;
    int interleaved;
    double mscale;
    int T, B, Hq, Hkv;
    int64_t Nmax;
    int d;
    void *q_out;
    void *K;
    void *V;
    uint8_t *codes;
    const int32_t *block_table;
    int64_t n_pages;
    int page_size;
    int max_pages;
    void *workspace;
    size_t workspace_bytes;
} adamas_rope_args;

int adamas_rope_append(const adamas_rope_args *args, adamas_stream_t stream);

/*
 * Causal attention of a chunk of new tokens over the whole cache (the new tokens'
 * rows are already in it).  Sequence b has n_b = cu_q[b + 1] - cu_q[b] new tokens,
 * the last n_b of its seq_lens[b] cached ones: query row i sits at slot
 * seq_lens[b] - n_b + i and sees slots 0 .. that one, softmax scale 1/sqrt(128).
 * n_b may be anything from 0 (the sequence is left out) over 1 (dense decode) to
 * the whole prompt.  A row whose slot is negative sees nothing: out 0, lse -inf.
 *   q    device bf16 [T][Hq][128]
 *   out  device bf16 [T][Hq][128]
 *   lse  device fp32 [T][Hq], optional: the natural logarithm of the row's sum of
 *        exp(score)
 * Scores, softmax statistics and output sums are fp32; the probabilities are
 * rounded to bf16 for their product with V (V is bf16 as well), the sum they are
 * divided by is not.  V rows are finite: a tile's masked products are 0 * V.
 * The same inputs give the same bits on every run.  K and V are at most 2^31 - 1
 * rows each (half a terabyte).
 */
typedef struct adamas_chunk_args {
    const void *q;
    const void *K;
    const void *V;
    const int32_t *cu_q;
    const int32_t *seq_lens;
    int T, B, Hq, Hkv;
    int64_t Nmax;
    int d;
    void *out;
    float *lse;
    float *mass;
    const int32_t *block_table;
    int64_t n_pages;
    int page_size;
    int max_pages;
    void *workspace;
    size_t workspace_bytes;
} adamas_chunk_args;

/* Bytes of device workspace adamas_chunk_attend needs (0: unsupported sizes). */
size_t adamas_chunk_workspace_bytes(int T, int B, int Hq, int Hkv, int d);

/* Uses every field but mass. */
int adamas_chunk_attend(const adamas_chunk_args *args, adamas_stream_t stream);

/*
 * mass[b][kvh][t] += sum over the chunk's rows that see slot t, and over the query
 * heads of kvh, of exp(q.K_t / sqrt(128) - lse[row]): the weight that slot t had in
 * the attention adamas_chunk_attend computed (lse as it wrote it).  To weigh the
 * tokens by a prompt's last rows only, pass those rows as the chunk.  Rows with
 * lse = -inf add nothing.  V and out are not used.
 */
int adamas_accumulate_chunk(const adamas_chunk_args *args, adamas_stream_t stream);

/*
 * The decode step's form: for every (b, query head) the softmax weights over the
 * kept tokens idx lists (as adamas_decode_step wrote them; entries outside
 * [0, seq_lens[b]) are skipped) are added to mass[b][kvh][idx].  idx is
 * [B][Hq][budget], or [B][Hkv][budget] with policy ADAMAS_SELECT_GROUP_SHARED (one
 * list for the query heads of a kv head).  Each list's tokens are distinct.
 */
typedef struct adamas_kept_args {
    const void *q;
    const void *K;
    const int32_t *idx;
    const int32_t *seq_lens;
    int B, Hq, Hkv;
    int64_t Nmax;
    int d;
    int budget;
    int policy;
    float *mass;
    const int32_t *block_table;
    int64_t n_pages;
    int page_size;
    int max_pages;
    void *workspace;
    size_t workspace_bytes;
} adamas_kept_args;

int adamas_accumulate_kept(const adamas_kept_args *args, adamas_stream_t stream);

/*
 * Eviction by accumulated attention weight.  For every (b, kv head) the
 * k_b = min(keep, seq_lens[b]) tokens of largest mass are kept -- equal masses: the
 * lower slot; -0 counts as 0, NaN as less than everything -- with the first n_sink
 * and the last n_recent tokens ranked ahead of all others (in slot order).  The kept
 * tokens move to slots 0 .. k_b - 1 in their old order: K, V, codes (optional) and
 * mass; mass from slot k_b on is set to 0 (a token appended there starts with no
 * weight).
 *   kept      device int32 [B][Hkv][keep]: their old slots, ascending, -1 past k_b
 *   new_lens  device int32 [B]: k_b; not seq_lens itself
 *   K_out ... mass_out, block_table_out, n_pages_out, page_size_out, max_pages_out,
 *             Nmax_out: the cache they move to, contiguous or paged; it must hold
 *             keep tokens per sequence and share no memory with the source (the
 *             rows of K_out past k_b are left as they were).  All NULL: in place, and no
 *             page may then be shared between sequences.
 */
typedef struct adamas_evict_args {
    void *K;
    void *V;
    uint8_t *codes;
    float *mass;
    const int32_t *seq_lens;
    int B, Hkv;
    int64_t Nmax;
    int d;
    int keep;
    int n_sink;
    int n_recent;
    int32_t *kept;
    int32_t *new_lens;
    const int32_t *block_table;
    int64_t n_pages;
    int page_size;
    int max_pages;
    void *K_out;
    void *V_out;
    uint8_t *codes_out;
    float *mass_out;
    int64_t Nmax_out;
    const int32_t *block_table_out;
    int64_t n_pages_out;
    int page_size_out;
    int max_pages_out;
    void *workspace;
    size_t workspace_bytes;
} adamas_evict_args;

int adamas_evict(const adamas_evict_args *args, adamas_stream_t stream);

/*
 * Synchronise `stream`, then copy the workspace's device error word into
 * *error_word (ADAMAS_DEVERR_* bits).  Returns ADAMAS_OK when the word is zero,
 * ADAMAS_ERR_DEVICE when it is not.
 */
int adamas_get_device_error(const void *workspace, size_t workspace_bytes, uint32_t *error_word,
                            adamas_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ADAMAS_H */
