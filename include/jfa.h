/*
 * jfa.h -- C ABI of the GB300 (sm_103a) Jagged Flash Attention library.
 *
 * Operation.  Exact softmax attention, forward and backward, computed directly on
 * variable-length sequences packed as jagged tensors (values plus int64 offsets),
 * never padded to the longest sequence, with an optional per-head additive bias and
 * unequal query and key/value lengths ("Jagged Flash Attention (JFA)", Definition).
 * "Exact" is the FlashAttention sense: tiling plus online softmax changes only the
 * rounding, never the function ("TLX-Optimized Jagged Flash Attention: Approaching
 * FA4-Level Performance on Blackwell", section "Why Jagged Flash Attention Deserves
 * Attention").  For sequence b, head h, local query row i < Lq_b and key j < Lk_b:
 *
 *   s_ij   = scale * q_i . k_j + beta_h(i, j)
 *   lse_i  = ln sum_j exp(s_ij)                 (over visible j)
 *   out_i  = sum_j exp(s_ij - lse_i) v_j
 *
 * with Lq_b = q_offsets[b+1] - q_offsets[b], Lk_b = kv_offsets[b+1] - kv_offsets[b].
 * Causal: key j is visible to query i iff j <= i + (Lk_b - Lq_b) (bottom-right
 * alignment; equal lengths give the usual j <= i).  A query row with no visible key
 * (Lk_b = 0, or causal with Lq_b > Lk_b) gets out = 0 and lse = -inf, and no gradient.
 * A row one of whose scores is NaN gets out = NaN and lse = NaN.
 *
 * Layout.  q, out, dout, dq: bf16 [total_q, H, d] row-major (token-major, heads
 * contiguous); k, v, dk, dv: bf16 [total_kv, H, d]; lse: fp32 [H, total_q];
 * offsets: int64 [B+1], offsets[0] = 0, non-decreasing, offsets[B] = total.  Empty
 * sequences are allowed.
 *
 * Ownership and execution.  Every pointer is a DEVICE pointer owned by the caller.
 * The library allocates nothing, keeps no state between calls (one process-wide
 * cache of driver entry points aside), and enqueues all work asynchronously on
 * `stream`.  Scratch memory is the caller's `workspace` (size from
 * jfa_workspace_size, 256-byte aligned, and its first 256 bytes zero before its first
 * use -- jfa_check_status keeps them so).  Calls sharing a workspace must not overlap.
 *
 * Errors.  Argument errors detectable on the host are returned synchronously and
 * enqueue nothing.  Errors found on the device (malformed offsets, a bounded
 * pipeline wait that ran out) are recorded in a status word in the workspace, the first
 * one sticking until jfa_check_status (which synchronises the stream) reads and clears
 * it.  On a device error the outputs of that call are unspecified.
 *
 * Requirements.  d in {64, 128}; H >= 1; B >= 1; every tensor pointer 16-byte
 * aligned; an sm_100-family GPU (built for sm_103a).
 */
#ifndef JFA_H_
#define JFA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* jfa_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
  JFA_OK = 0,
  JFA_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned pointer */
  JFA_ERR_UNSUPPORTED = 2, /* head_dim not in {64,128}, unsupported bias kind or bias gradient */
  JFA_ERR_WORKSPACE = 3,   /* workspace missing, too small or misaligned; device: one that the cache attention
                              cannot use until it is zeroed */
  JFA_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed (launch, tensor-map encode) */
  JFA_ERR_BAD_OFFSETS = 5, /* device: offsets not 0-based, not monotone, or last != total (also kind-2 bias block offsets) */
  JFA_ERR_TIMEOUT = 6,     /* device: a bounded pipeline wait ran out; outputs unspecified */
  JFA_ERR_BAD_PAGES = 7,   /* device: a page table entry that a call needs is not a page of the cache, or a
                              token lies past the table's last page */
  JFA_ERR_NO_PAGES = 8     /* device: fewer free pages than a reservation needs; none were taken */
} jfa_status;

/* Additive attention bias (the user-defined biases of "Jagged Flash Attention
 * (JFA)", Definition).  kind 0 = none.  kind 2 = general jagged bias (below).
 * kind 1 = per-head relative-position table:
 *   beta_h(i, j) = table[h * num_buckets + clamp(j - i + center, 0, num_buckets - 1)]
 * with i, j local 0-based positions; added after scaling.  `table` is a device
 * fp32 [H][num_buckets] array; num_buckets in [1, 8192].
 * `grad` (kind 1, jfa_backward only; NULL = not wanted): a device fp32 [H][num_buckets]
 * array, 4-byte aligned, not overlapping any other argument, that jfa_backward
 * overwrites with the gradient of sum(dout * out) w.r.t. `table`: entry (h, n) is the sum
 * of dS_ij = P_ij (dP_ij - D_i) over every sequence's visible pairs (i, j) whose bucket is
 * n.  It is accumulated with fp32 additions in L2 whose order is not fixed, so repeated
 * calls can differ in the last bits.  jfa_forward ignores it.
 * kind 2 = general jagged bias: beta_h(i, j) = values[h * plane + block_offsets[b] +
 * i * round_up(Lk_b, 8) + j], i.e. one Lq_b x Lk_b matrix per sequence and head, stored
 * row-major with each row padded to a multiple of 8 elements (the padding is never
 * read), the blocks of one head packed into a plane of `plane` elements.  `values` is a
 * device bf16 array [H][plane], 16-byte aligned; `block_offsets` a device int64 array
 * [B+1] with block_offsets[0] = 0 and block_offsets[b+1] - block_offsets[b] =
 * Lq_b * round_up(Lk_b, 8), block_offsets[B] = plane -- checked on the device (a mismatch
 * is JFA_ERR_BAD_OFFSETS and no attention is computed).  Added after scaling, like kind 1.
 * `grad` must be NULL for kind 2; its gradient goes to `values_grad` instead (jfa_backward
 * only; NULL = not wanted): a device bf16 array with the layout of `values`, 16-byte
 * aligned, not overlapping any other argument, overwritten with dS_ij = P_ij (dP_ij - D_i)
 * at each block element (0 for pairs the causal mask hides and for the row padding). */
typedef struct {
  int kind;
  const float* table;
  int num_buckets;
  int center;
  float* grad;
  const void* values;            /* kind 2 */
  const int64_t* block_offsets;  /* kind 2 */
  int64_t plane;                 /* kind 2 */
  void* values_grad;             /* kind 2, jfa_backward */
} jfa_bias;

/* Bytes of workspace jfa_forward (is_backward = 0) or jfa_backward (is_backward = 1)
 * needs for these sizes.  Returns 0 on invalid sizes. */
size_t jfa_workspace_size(int B, int H, int d, int64_t total_q, int64_t total_kv, int is_backward);

/* Forward.  Writes out (bf16 [total_q, H, d]) and lse (fp32 [H, total_q], natural
 * log of the row's sum of exp(s_ij)).  bias may be NULL. */
jfa_status jfa_forward(const void* q, const void* k, const void* v, const int64_t* q_offsets,
                       const int64_t* kv_offsets, int B, int H, int d, int64_t total_q, int64_t total_kv,
                       const jfa_bias* bias, float scale, int causal, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, jfa_stream_t stream);

/* Backward of sum(dout * out) w.r.t. q, k, v (the backward pass listed among JFA's
 * features, "Jagged Flash Attention (JFA)", Definition; split scheme of "Four generations"
 * item 2: dK/dV computed per key/value block, dQ in a separate pass that owns each
 * dQ tile, no atomics).  out and lse must be the forward's results for the same
 * inputs.  dq, dk, dv are bf16 with the shapes of q, k, v and are fully overwritten
 * (rows of keys no query sees get 0).  With a relative-position bias whose `grad` is
 * non-NULL, the table's gradient is written there too (see jfa_bias). */
jfa_status jfa_backward(const void* dout, const void* q, const void* k, const void* v, const void* out,
                        const float* lse, const int64_t* q_offsets, const int64_t* kv_offsets, int B, int H,
                        int d, int64_t total_q, int64_t total_kv, const jfa_bias* bias, float scale,
                        int causal, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                        jfa_stream_t stream);

/* ---- Sliding window with sinks, key/value heads shared by groups of query heads.
 *
 * The same attention, causal, with query i of a sequence (at position p = i + Lk_b - Lq_b)
 * seeing key j iff  j <= p  and  (j > p - window  or  j < sinks):  the last `window` keys up to
 * its own position, and the sequence's first `sinks` keys always.  A window of at least Lk_b is
 * plain causal attention.  Query head h reads key/value head h / (H / H_kv).  A row that sees no
 * key (p < 0) gets out = 0, lse = -inf and no gradient.
 *
 * q, out, dout, dq: bf16 [total_q, H, d]; k, v, dk, dv: bf16 [total_kv, H_kv, d]; the rest as for
 * jfa_forward / jfa_backward.  H a multiple of H_kv; window >= 1; sinks in 0 .. 128.  Cost goes
 * with the visible key tiles, not with the sequence length squared.  Keys that no query of their
 * sequence sees (when queries follow a longer history) are not read: they may hold anything,
 * NaN included, and get zero gradients.  A non-finite value in a key or value that some query
 * sees, or in dout, may reach every row of that sequence and head, in out and in the gradients.  A
 * row one of whose scores is NaN (or +inf) gets out = NaN and lse = NaN; lse = -inf means that it
 * sees no key (or that all its scores are -inf).  Outputs must not overlap inputs or one another
 * (equal pointers are refused), but out may be q, and dq may be q, dout or out.  dk and dv sum over
 * the group's query heads in fp32, in a fixed order (results are bit-reproducible). */
size_t jfa_window_workspace_size(int B, int H, int H_kv, int d, int64_t total_q, int64_t total_kv, int sinks,
                                 int is_backward);
jfa_status jfa_window_forward(const void* q, const void* k, const void* v, const int64_t* q_offsets,
                              const int64_t* kv_offsets, int B, int H, int H_kv, int d, int64_t total_q, int64_t total_kv,
                              int window, int sinks, float scale, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, jfa_stream_t stream);
jfa_status jfa_window_backward(const void* dout, const void* q, const void* k, const void* v, const void* out,
                               const float* lse, const int64_t* q_offsets, const int64_t* kv_offsets, int B, int H,
                               int H_kv, int d, int64_t total_q, int64_t total_kv, int window, int sinks, float scale,
                               void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                               jfa_stream_t stream);

/* Forward without a workspace, for callers that cannot allocate device memory.  The
 * pages have no counterpart to this entry point.  Hosts such as inference-runtime
 * plugins and services on a fixed, pre-planned memory arena give a kernel library
 * only its inputs and outputs and must not call cudaMalloc on their hot path (it can
 * synchronise the device and breaks the arena's budget); this call runs jfa_forward
 * with its scratch in a file-scope device array of 9 MiB that every GPU loading the
 * library holds until exit.  Arguments and results are those of jfa_forward.
 * - Sizes whose workspace (jfa_workspace_size(..., 0)) exceeds 9 MiB are rejected with
 *   JFA_ERR_WORKSPACE before anything is enqueued.
 * - The first call on a device looks up the array's device address (cudaGetSymbolAddress)
 *   with that device current; make that first call before any stream capture.
 * - Allocates nothing: no cudaMalloc, cudaFree or allocating library routine.
 * - Every call on a device shares the one array: calls whose work overlaps on the GPU
 *   (e.g. on two streams) race and must be serialised by the caller.  Each call
 *   rewrites all of the scratch it reads, so no clearing is needed between calls.
 * - Device-detected errors (bad offsets, wait timeout) land in the shared array and are
 *   not reported to the caller; use jfa_forward with a workspace to read them. */
jfa_status jfa_forward_noalloc(const void* q, const void* k, const void* v, const int64_t* q_offsets,
                               const int64_t* kv_offsets, int B, int H, int d, int64_t total_q, int64_t total_kv,
                               const jfa_bias* bias, float scale, int causal, void* out, float* lse,
                               jfa_stream_t stream);

/* ---- Paged key/value cache: serving one new token at a time.
 *
 * k, v: bf16 [num_pages][H_kv][page_size][d], the caller's, 16-byte aligned; token p of
 * sequence b lives in row p % page_size of page page_table[b * max_pages + p / page_size].
 * page_size in {16, 32, 64, 128}; d in {64, 128}; num_pages * H_kv * page_size < 2^31 and
 * max_pages * page_size <= 2^31 - 128.  page_table: device int32 [B][max_pages]; entries that a
 * call does not need may hold anything.  lengths: device int32 [B], tokens of each
 * sequence.  Pages may be shared by sequences for reading. */
typedef struct {
  void* k;
  void* v;
  int64_t num_pages;
  int H_kv, page_size, d;
  const int32_t* page_table;
  int max_pages;
  const int32_t* lengths;
  int B;
} jfa_cache;

/* Bytes of workspace jfa_cache_attention and jfa_qcache_attention need (the appends, jfa_pages_reserve and
 * jfa_pages_release need the first 256 of them); 256-byte aligned, zero before its first use, every call
 * leaves what it needs zero, zero again.  One workspace serves all these calls, at any sizes that it is
 * large enough for, but only one call at a time.  When forward or backward calls of this library have used it, or after a
 * JFA_ERR_TIMEOUT, zero it again: as long as its counters may not be zero, the attentions
 * compute nothing and report JFA_ERR_WORKSPACE.  (The other calls need no zeroing.)  Returns 0
 * on invalid sizes. */
size_t jfa_cache_workspace_size(int B, int H, int H_kv, int d);

/* Append new tokens, keys rotated by their position on the way.  Sequence b's new tokens are
 * rows [offsets[b], offsets[b+1]) of k and v (device int64 [B+1], offsets[0] = 0,
 * non-decreasing, offsets[B] <= total: rows behind the last sequence are neither read nor
 * written), and take positions lengths[b], lengths[b] + 1, ...  Rows of a token are H_kv
 * (q: H) heads of d contiguous bf16; tokens k_stride (v_stride, q_stride) elements apart, so
 * that slices of one fused projection can be given; 16-byte aligned, strides multiples of 8.
 *
 * Rotation: the first rot_dim (0 .. d, a multiple of 16) elements of each head of k (and q)
 * form rot_dim / 2 pairs, pair i = (x_i, x_{i + rot_dim/2}), or (x_2i, x_2i+1) when
 * `interleaved`, and (a, b) becomes (a cos t - b sin t, b cos t + a sin t) with
 * t = position * frequencies[i]; `frequencies` is a HOST array of rot_dim / 2 doubles
 * (radians per position), read during the call.  At any position sines and cosines are good to
 * 2^-22 of their value and 2^-32 of a turn, frequencies up to 2^20 taken as exact.  Results are rounded
 * to bf16 once.
 *
 * q (may be NULL) is rotated into q_out, contiguous [total][H][d]; with k_out non-NULL the
 * rotated keys are also written there, contiguous [total][H_kv][d] (for the prompt's own
 * attention).  q_out may be q and k_out may be k when those are contiguous;
 * other overlaps of outputs with inputs or one another are not allowed (equal pointers are refused).  lengths_out (may
 * be NULL): device int32 [B], overwritten with lengths[b] + the number of appended tokens; it
 * may be `lengths` itself.  Each cache row must be written by one token only.
 *
 * Errors on the device: malformed offsets or a negative length (JFA_ERR_BAD_OFFSETS); a token
 * whose page is missing (JFA_ERR_BAD_PAGES; that token is not stored).  After an error
 * lengths_out[b] is lengths[b] for a sequence with a negative length or a token that was not stored
 * (the call may be repeated for it), and for all sequences when the offsets are malformed; the
 * others advance. */
jfa_status jfa_cache_append(const jfa_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const void* q, int64_t q_stride, int H, const int64_t* offsets, int64_t total,
                            const double* frequencies, int rot_dim, int interleaved, void* q_out, void* k_out,
                            int32_t* lengths_out, void* workspace, size_t workspace_bytes, jfa_stream_t stream);

/* Attention of each sequence's newest token over the cache: q, out bf16 [B][H][d], lse fp32
 * [H][B]; H a multiple of H_kv, query head h reading key/value head h / (H / H_kv).  With
 * L = lengths[b] (the newest token, at position L - 1, already appended), key j is visible iff
 * j < L and (j >= L - window or j < sinks); window >= 1, sinks >= 0.  L = 0 gives out = 0 and
 * lse = -inf.  Only pages that hold a visible key are looked up, and what rows hold that show
 * no key does not matter (NaN included); a NaN among its scores gives a head out = NaN and
 * lse = NaN.  A length below 0 or above max_pages * page_size is
 * JFA_ERR_BAD_OFFSETS, a visible key on a page outside the cache JFA_ERR_BAD_PAGES. */
jfa_status jfa_cache_attention(const jfa_cache* cache, const void* q, int H, int window, int sinks, float scale,
                               void* out, float* lse, void* workspace, size_t workspace_bytes, jfa_stream_t stream);

/* ---- The same cache held in 8 bits.
 *
 * cache.k and cache.v hold codes of one byte, [num_pages][H_kv][page_size][d], e4m3 or int8 as `kind` says; the
 * `block` tokens of an aligned block of a page (16, 32, 64 or 128, at most page_size) and head share a scale in
 * k_scale / v_scale, fp32 [num_pages][H_kv][page_size / block], the caller's.  A value is code * scale.  All
 * else is as for jfa_cache. */
enum { JFA_CODES_E4M3 = 0, JFA_CODES_INT8 = 1 };
typedef struct {
  jfa_cache cache;
  float* k_scale;
  float* v_scale;
  int block;
  int kind;
} jfa_qcache;

/* jfa_cache_append into such a cache: arguments, rotation, other outputs, lengths and errors are the same.
 * Keys are rotated in fp32 and rounded to codes once (k_out: to bf16 once).  A block's scale is the smallest
 * power of two, 2^-126 at least, with which the largest code (448, 127) holds the block's new values, or sqrt(2)
 * times the largest element of the block's new keys where keys are rotated; or the scale it has, where tokens
 * of the block that came before these have a larger one (one of another origin may be negative: its magnitude
 * counts).  When it grows, the codes of those are rounded again (int8 codes may be -128): a block is one sequence's
 * to append to, only whole blocks may be shared.  Codes are to the nearest
 * of value / scale, ties to even (by a scale of another origin that is no power of two: of value times 1 / scale
 * in fp32).  Where a new value of a block and head is not finite, the block's scale
 * becomes NaN, and stays so until its first token is written again.  (Powers of two cost e4m3 nothing but range;
 * of int8 a code's step is up to 2, with rotated keys 2 sqrt(2), times the block's largest |x| / 127.)  Workspace: 256 bytes, as there. */
jfa_status jfa_qcache_append(const jfa_qcache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const void* q, int64_t q_stride, int H, const int64_t* offsets, int64_t total,
                             const double* frequencies, int rot_dim, int interleaved, void* q_out, void* k_out,
                             int32_t* lengths_out, void* workspace, size_t workspace_bytes, jfa_stream_t stream);

/* jfa_cache_attention over such a cache, with scales of any origin and value: the same arguments, mask, results
 * and errors, and the same workspace (jfa_cache_workspace_size).  What codes and scales hold that show no key
 * does not matter.  Products and sums run on the codes as they are; the weights of the values are rounded to
 * f16 (2^-11 relative; those that are below 2^-21 of the largest, or of 2^-126, with their scales, to 2^-32 of that).
 * Scores are fp32 products of a head's factor, its largest |q| to a power of two times scale, and the key's scale: a
 * factor below 2^-112 has fewer bits, which counts where key scales are above 2^90.  A NaN in a visible key's codes
 * or scale gives its head out = NaN and lse = NaN, one in a value's out = NaN.  out may be q. */
jfa_status jfa_qcache_attention(const jfa_qcache* cache, const void* q, int H, int window, int sinks, float scale,
                                void* out, float* lse, void* workspace, size_t workspace_bytes, jfa_stream_t stream);

/* ---- Pages for either cache, on the device.
 *
 * A sequence with L tokens holds ceil(L / page_size) pages, the first entries of its row of page_table (device
 * int32 [B][max_pages]).  free_pages: device int32 [num_pages], of which the first *free_count (device int32)
 * are pages that nobody holds.  page_size in {16, 32, 64, 128}; B <= 2^30; max_pages * page_size
 * <= 2^31 - 128.  Results do not depend on timing.  Workspace: the first 256 bytes of a cache's, as for jfa_cache_append.
 *
 * jfa_pages_reserve takes the pages that offsets[b+1] - offsets[b] new tokens of each sequence need behind its
 * lengths[b]: from the list's end, sequences in order, positions in order (page i of them is
 * free_pages[*free_count - 1 - i]), and writes them into the table.  slots (may be NULL): device int64 [total],
 * for each new token's row page * page_size + its row in the page, -1 for rows behind the last sequence.
 * free_count_out (may be free_count) becomes the pages left.  free_pages and lengths stay as they are (an append
 * advances the lengths).  offsets as for jfa_cache_append.
 * Errors on the device, none of which takes a page (slots are then -1): offsets, a length or *free_count out of
 * range (JFA_ERR_BAD_OFFSETS), a token past the table's last page (JFA_ERR_BAD_PAGES), too few free pages
 * (JFA_ERR_NO_PAGES).  A token on a page outside 0 .. num_pages - 1 gets slot -1 (JFA_ERR_BAD_PAGES). */
jfa_status jfa_pages_reserve(int32_t* page_table, int B, int max_pages, int page_size, const int32_t* lengths,
                             const int64_t* offsets, int64_t total, const int32_t* free_pages, int64_t num_pages,
                             const int32_t* free_count, int32_t* free_count_out, int64_t* slots, void* workspace,
                             size_t workspace_bytes, jfa_stream_t stream);

/* jfa_pages_release puts the pages back that sequences no longer need when only their first keep[b] tokens stay
 * (device int32 [B], 0 .. lengths[b]): behind the list's end, sequences in order, positions in order.
 * free_count_out (may be free_count) becomes the pages on the list, lengths_out (may be lengths) keep.  The table
 * stays as it is.  A page that several sequences hold must be put back once only: by those that share it, keep
 * what is shared.  Errors on the device, none of which puts a page back or changes a length: a length, keep or
 * *free_count out of range (JFA_ERR_BAD_OFFSETS), more pages than the list has room for (JFA_ERR_BAD_PAGES).  A
 * table entry that is no page is put on the list all the same, and reported (JFA_ERR_BAD_PAGES). */
jfa_status jfa_pages_release(const int32_t* page_table, int B, int max_pages, int page_size, const int32_t* lengths,
                             const int32_t* keep, int32_t* free_pages, int64_t num_pages, const int32_t* free_count,
                             int32_t* free_count_out, int32_t* lengths_out, void* workspace, size_t workspace_bytes,
                             jfa_stream_t stream);

/* Synchronises `stream`, then returns the first device-side error recorded in
 * `workspace` since the previous jfa_check_status (JFA_OK if none; else JFA_ERR_BAD_OFFSETS,
 * JFA_ERR_TIMEOUT, JFA_ERR_WORKSPACE, JFA_ERR_BAD_PAGES or JFA_ERR_NO_PAGES) and clears it. */
jfa_status jfa_check_status(void* workspace, jfa_stream_t stream);

/* Static, NUL-terminated description of a status code. */
const char* jfa_status_string(jfa_status s);

/* Number of kernels the last successful jfa_forward / jfa_backward call on this
 * thread enqueued (for launch accounting). */
int jfa_last_launch_count(void);

/* Description of the last failed CUDA runtime/driver call made by this library on the
 * calling thread (the cause behind a JFA_ERR_CUDA); "" if none.  Thread-local, static. */
const char* jfa_last_error(void);

/* Kernel kinds for per-kernel timing.  (A windowed call's kernels count as the plain call's of
 * their role, an 8-bit cache's as the bf16 cache's; the join, cache and page kinds, and the windowed backward passes at d = 64, record no
 * developer trace.) */
enum { JFA_KERNEL_PLAN = 0, JFA_KERNEL_FORWARD = 1, JFA_KERNEL_BWD_PREPROCESS = 2, JFA_KERNEL_BWD_DKDV = 3,
       JFA_KERNEL_BWD_DQ = 4, JFA_KERNEL_BWD_FUSED = 5, JFA_KERNEL_BWD_NSP = 6, JFA_KERNEL_BWD_JOIN = 7,
       JFA_KERNEL_CACHE_APPEND = 8, JFA_KERNEL_CACHE_ATTENTION = 9, JFA_KERNEL_CACHE_PAGES = 10,
       JFA_NUM_KERNEL_KINDS = 11 };

/* Benchmark support (not part of the attention itself).  While enabled (process-wide),
 * every kernel launch is bracketed by two CUDA events recorded on the launch stream.
 * jfa_timing_read waits for the recorded events, adds each kernel's elapsed time (ms)
 * to ms[kind] and its launch count to launches[kind] for kind < n_kinds, then drops
 * the records.  Both return JFA_ERR_CUDA if an event call fails. */
jfa_status jfa_timing_enable(int on);
jfa_status jfa_timing_read(double* ms, int* launches, int n_kinds);

/* Failure-detection self test (not part of the attention itself).  Enqueues one tiny
 * kernel whose single thread waits on a pipeline barrier that nothing ever signals,
 * through the bounded wait every kernel of this library uses; after `timeout_ns`
 * (1 ns .. 2 s) the wait gives up and JFA_ERR_TIMEOUT is recorded in the workspace
 * status word, readable with jfa_check_status.  Nothing faults or hangs; the context
 * stays usable.  `workspace` needs 256 bytes (zeroed status word). */
jfa_status jfa_selftest_wait_timeout(void* workspace, uint64_t timeout_ns, jfa_stream_t stream);

/* Which backward pass takes a sequence of two or more query tiles (128 rows each), for
 * every later jfa_backward call in the process.  Sequences of 2 .. max_tiles query tiles
 * take the non-sequence-parallel pass -- one CTA owns a (sequence, head), forms every tile
 * pair's S, P, dP and dS once and computes dK, dV and dQ from them (five GEMMs per tile
 * pair), summing dQ over key tiles in an fp32 buffer in the workspace with one writer per
 * row ("Jagged Flash Attention (JFA)", "Four generations" item 2, the reading in which
 * the backward is not parallel over a sequence's query tiles); longer sequences take the
 * split passes (dK/dV per key tile, then dQ per query tile: seven GEMMs per tile pair, no
 * sum buffer).  max_tiles in 0 .. 16; below 2 every such sequence takes the split passes
 * (the default, which measured faster on GB300) and jfa_backward launches five kernels, not
 * the pass's sixth.  Both paths give the same results within
 * rounding and are each deterministic.  With max_tiles >= 2 the backward workspace also
 * holds the fp32 dQ sums (4 * total_q * H * d more bytes): jfa_workspace_size reflects the
 * setting at the time it is called, and a workspace sized before the pass was enabled is
 * rejected with JFA_ERR_WORKSPACE.  A negative max_tiles only reads the setting.
 * Returns the previous setting, or -1 (nothing changed) for max_tiles > 16. */
int jfa_set_nsp_max_tiles(int max_tiles);

/* The item hand-off wait limit, in ns, that the kernels use for a launch whose planner
 * found `planned_tile_pairs` 128x128 (query tile, key tile) pairs over all heads, to be
 * shared by `ctas` persistent CTAs, the costliest single work item being
 * `max_item_tile_pairs` pairs (not part of the attention itself; exported so the rule can
 * be checked without a GPU).  A CTA's scheduler waits for its previous items to finish
 * before it claims the next, and its roles wait for the next item to be claimed: such a
 * wait lasting longer ends the CTA with JFA_ERR_TIMEOUT.  The limit is 2 s plus 32 us for
 * each pair of one CTA's share (rounded up) and of the costliest item, capped at 2 s + 1 h;
 * negative arguments count as 0, `ctas` < 1 as 1.  32 us is about 30 times the time one SM
 * takes for a pair, so no hand-off of a correct launch comes near it, whatever the
 * launch's size.  (Waits inside an item's tile pipeline last at most a few tiles' time and
 * keep a fixed 2 s limit.) */
uint64_t jfa_wait_limit_ns(int64_t planned_tile_pairs, int ctas, int64_t max_item_tile_pairs);

/* Developer tracing (not part of the attention itself).  With a non-NULL device buffer,
 * kernels of `kernel_kind` (JFA_KERNEL_*) launched afterwards record the pipeline events
 * of their first CTA: uint64 entries (SM clock << 16 | role << 8 | event id) in five
 * regions of bytes/40 entries, one per warp role (0 streaming TMA producer, 1 MMA issuer,
 * 2 and 3 the two compute warpgroups, 4 resident-tile loader); each launch overwrites
 * them; unused entries are left as they were.  A NULL buffer or a kind outside [0, JFA_NUM_KERNEL_KINDS) turns tracing off.
 * Process-wide; returns JFA_ERR_INVALID_ARG for a buffer too small or not 8-byte aligned. */
jfa_status jfa_trace_configure(void* device_buffer, size_t bytes, int kernel_kind);

#ifdef __cplusplus
}
#endif
#endif /* JFA_H_ */
