/*
 * tq.h -- C ABI of the B200 TurboQuant packed-KV library (libtq.so).
 *
 * Two operations make up the hot path:
 *
 *   tq_quantize_append  rotate each K/V row with a randomized Hadamard transform,
 *                       store its fp32 L2 norm, Lloyd-Max-encode every rotated unit
 *                       coordinate and bit-pack the codes into the row's page slot;
 *   tq_paged_decode     one attention decode step straight over the packed pages:
 *                       rotate q once, score each key on its codes, online softmax,
 *                       accumulate V in the rotated domain, inverse-rotate the output.
 *
 * Sources (page title, section):
 *   TorbuQuant (ginkgoq.github.io/TurboQuant), "TQ4 page tensor" diagram -- page
 *     tensor [num_blocks, block_size, num_kv_heads, slot_bytes], slot -> (block, row),
 *     slot = [K: packed indices, fp32 norm][V: packed indices, fp32 norm],
 *     K bytes ceil(D*k_bits/8)+4, V bytes ceil(D*v_bits/8)+4, optional padding;
 *     the stages "Quantize: rotate, normalize, codebook-encode, pack" and "Store".
 *   tq-kv (shadowgraph.io), "How It Works" step 3 (randomized Hadamard transform)
 *     and "Library API" (generate_signs(dim, seed), pre_rotate_query_with_signs,
 *     fused_attention_scores on compressed keys); "Custom CUDA Kernel Stack"
 *     (flash decode with split-KV and online softmax; attention score without
 *     decompression).
 *   turboquant_serve 0.1.2, "Architecture" (update(): rotate, normalize,
 *     Lloyd-Max encode, bit-pack; _decode(): unpack, decode, restore magnitude,
 *     rotate back; one rotation per head_dim; codebooks fitted once and shared).
 *   turboquant_pro 1.4.2, "How It Works" (norm preserved alongside the bits;
 *     8 x 3-bit = 3 bytes) and "Fused CUDA decode" (split-K decode on the codes).
 *
 * Conventions where the pages are silent (the library and its tests agree on them):
 *   - signs: s_j = -1 if bit 63 of the j-th SplitMix64 output seeded with
 *     sign_seed is set, else +1 (j = 0..D-1); the same signs serve K, V, q and
 *     every head; rotation y = (1/sqrt(D)) H (s * x), H the natural-order
 *     (Sylvester) Hadamard matrix;
 *   - norm: L2 norm of the input row, stored as fp32 (rows of any finite magnitude;
 *     a norm beyond the fp32 range stores +inf); unit coordinates u = y / n;
 *   - code: idx = number of boundaries b_i with b_i < u (ties to the lower cell);
 *     a zero row stores norm 0 and codes idx(0); a row holding a non-finite value
 *     stores codes 0 and a quiet-NaN norm (0x7FC00000) and raises
 *     TQ_DEVERR_NONFINITE;
 *   - packing: code j fills bits [j*bits, (j+1)*bits) of a little-endian bit
 *     stream (bit p = bit p%8 of byte p/8); the fp32 norm follows, little endian;
 *   - GQA: query head h reads KV head h / (H_q / H_kv).
 *
 * Memory: every pointer below is a DEVICE pointer unless stated otherwise.  The
 * caller owns all buffers.  Calls are asynchronous on `stream` (a cudaStream_t
 * passed as void*, NULL = legacy default stream); host-side validation errors are
 * returned synchronously and nothing is enqueued.  Errors found by a kernel (an
 * out-of-range slot or block id, a non-finite input row) are OR-ed into a
 * per-device error word read by tq_get_device_error(); the offending row or
 * block is skipped, nothing faults.
 */
#ifndef TQ_H_
#define TQ_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define TQ_API __attribute__((visibility("default")))
#else
#define TQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TQ_OK = 0,
  TQ_ERR_INVALID_ARG = 1,  /* bad pointer, shape, stride, dtype or parameter   */
  TQ_ERR_UNSUPPORTED = 2,  /* valid but not built: head_dim, bits or GQA group */
  TQ_ERR_CUDA = 3,         /* a CUDA runtime call failed (launch, memcpy, ...)  */
  TQ_ERR_DEVICE = 4,       /* a kernel reported an error (see the error word)  */
  TQ_ERR_WORKSPACE = 5     /* workspace missing or too small                    */
} tq_status;

typedef enum {
  TQ_U8 = 0,
  TQ_I32 = 1,
  TQ_I64 = 2,
  TQ_F32 = 3,
  TQ_BF16 = 4,
  TQ_F16 = 5
} tq_dtype;

/* Device error word bits (tq_get_device_error). */
#define TQ_DEVERR_SLOT_RANGE 0x1    /* slot_mapping entry >= num_blocks*block_size */
#define TQ_DEVERR_BLOCK_RANGE 0x2   /* block_table entry outside [0, num_blocks)   */
#define TQ_DEVERR_NONFINITE 0x4     /* a K/V input row held a NaN or an infinity   */
#define TQ_DEVERR_SEQLEN_RANGE 0x8  /* seq_len < 0 or > max_blocks*block_size      */
#define TQ_DEVERR_TIMEOUT 0x10      /* a bounded wait inside a kernel gave up        */
#define TQ_DEVERR_LAYOUT 0x20       /* the decode kernel's shared-memory layout did not
                                       match its launch; the launch did nothing      */
#define TQ_DEVERR_NO_PAGES 0x40     /* too few free pages: a resize or fork was refused */
#define TQ_DEVERR_SEQ_INDEX 0x80    /* tq_pages_fork: a sequence index outside [0, B), a
                                       child named twice or not empty, a bad length   */

/* A strided view of a device array.  Strides are in ELEMENTS; shape[i] and
 * stride[i] for i >= ndim are ignored.  data must be aligned to the element size. */
typedef struct {
  void* data;
  int32_t dtype;      /* tq_dtype */
  int32_t ndim;
  int64_t shape[4];
  int64_t stride[4];
} tq_tensor;

/* One fp32 Lloyd-Max table (Beta-sphere density for `dim`): `centroids` holds
 * 2^bits ascending values, `boundaries` the 2^bits - 1 ascending cell edges.
 * Both are device pointers, 4-byte aligned, owned by the caller and read by
 * every launch ("fitted once ... and shared", turboquant_serve, "Codebook sharing"). */
typedef struct {
  int32_t dim;
  int32_t bits;
  const float* centroids;
  const float* boundaries;
} tq_codebook;

typedef struct {
  tq_codebook k;
  tq_codebook v;
} tq_codebooks;

/* The dense random rotation R (turboquant_serve 0.1.2, "Architecture" and "Rotation": a
 * fixed random orthogonal matrix, seeded by head_dim; TorbuQuant, "Current Status": QR
 * rotation) as two bf16 matrices: R = hi + lo, [dim][dim] row-major (row j gives output
 * coordinate j), bf16 bit patterns in device memory, 16-byte aligned, owned by the caller.
 * The library's data files rotations/qr_d<D>.tqrt hold them (hi = bf16 of the seeded
 * Haar matrix, lo = bf16 of the remainder; R is exact in fp32 and orthogonal to ~1e-5). */
typedef struct {
  int32_t dim;
  const uint16_t* hi;
  const uint16_t* lo;
} tq_rotation;

/* Bytes of one slot before padding: (ceil(D*k_bits/8)+4) + (ceil(D*v_bits/8)+4)
 * (TorbuQuant, "TQ4 page tensor").  Host only; *out receives the value.
 * Errors: TQ_ERR_INVALID_ARG for dim < 1, bits outside 1..8 or out == NULL. */
TQ_API tq_status tq_slot_bytes(int32_t dim, int32_t k_bits, int32_t v_bits, int32_t* out);

/* Quantize-append (TorbuQuant "Quantize" and "Store"; turboquant_serve update()).
 *
 *   pages        u8  [num_blocks, block_size, H_kv, slot_stride]; the last dim is
 *                contiguous, slot_stride >= tq_slot_bytes(D, k_bits, v_bits) and a
 *                multiple of 8; bytes beyond slot_bytes are never written.
 *   slot_mapping i64 [T]: token t goes to slot s = slot_mapping[t], i.e.
 *                page[s / block_size, s % block_size, h, :] for every KV head h;
 *                s < 0 skips the token; s >= num_blocks*block_size skips it and
 *                raises TQ_DEVERR_SLOT_RANGE.
 *   k, v         [T, H_kv, D] in bf16, f16 or f32 (same dtype); the last dim is
 *                contiguous; rows are read exactly (converted to fp32).
 *   cb           host pointer to the K and V tables (device arrays inside);
 *                cb->k.dim == cb->v.dim == D, cb->k.bits == k_bits, cb->v.bits == v_bits.
 *   sign_seed    SplitMix64 seed of the rotation signs.
 *   k_bits, v_bits  1..8.  D must be 64, 128 or 256.
 * Two tokens mapped to the same slot race (either row may win).
 * Two launches: the fast path, then a redo that returns at once unless some row's sum
 * of squares left the fast path's range (rows of magnitude beyond about 1e14 or below
 * about 1e-10, zero rows, non-finite rows), in which case the whole call is done again
 * with an exact power-of-two rescaling of those rows.  The two share a per-device flag:
 * calls on one device whose kernels overlap on the GPU (unordered streams) must be
 * ordered.
 * Fast paths (same results, chosen per call on the host):
 *   - k and v are staged by tensor copies when they are 16-bit, 16-byte aligned with
 *     token and head strides that are multiples of 8 elements, and H_kv divides
 *     2048/D or is a multiple of it;
 *   - each token's slots are stored with one bulk copy when, in addition to that H_kv
 *     rule, slot_stride == tq_slot_bytes(...), pages is 16-byte aligned with block and
 *     row strides that are multiples of 16, and the token's run of slots is a
 *     multiple of 16 bytes;
 *   - otherwise, when pages is 16-byte aligned with block, row and head strides that
 *     are multiples of 16 (a padded slot_stride), each slot's first
 *     (slot_bytes & ~15) bytes are stored by one bulk copy and the rest by 4-byte
 *     stores; the padding is not written.
 *   Other layouts take lane-wise copies.
 * Errors: TQ_ERR_INVALID_ARG / TQ_ERR_UNSUPPORTED (nothing enqueued), TQ_ERR_CUDA. */
TQ_API tq_status tq_quantize_append(tq_tensor pages, tq_tensor slot_mapping, tq_tensor k,
                             tq_tensor v, const tq_codebooks* cb, uint64_t sign_seed,
                             int32_t k_bits, int32_t v_bits, void* stream);

/* Paged decode (tq-kv "Library API" fused scores on compressed keys; "Custom CUDA
 * Kernel Stack" flash decode v2 split-KV with online softmax; turboquant_pro
 * "Fused CUDA decode").
 *
 *   out          [B, H_q, D], f32 or the dtype of q; last dim contiguous.
 *                out[b, h] = sum_t softmax_t(scale * <q[b,h], k_hat_t>) v_hat_t over
 *                t < seq_lens[b], where k_hat/v_hat are the dequantized rows
 *                norm * R^T c[idx] of KV head h / (H_q/H_kv).  seq_lens[b] == 0 gives 0.
 *   q            [B, H_q, D] in bf16, f16 or f32; last dim contiguous.
 *   pages        as in tq_quantize_append (k_bits/v_bits taken from cb).
 *   block_table  i32 [B, max_blocks]: token t of sequence b lives in block
 *                block_table[b, t / block_size], row t % block_size.  Entries past
 *                the sequence are not read.  An entry outside [0, num_blocks) raises
 *                TQ_DEVERR_BLOCK_RANGE and its block is skipped.
 *   seq_lens     i32 [B]; 0 <= seq_lens[b] <= max_blocks * block_size, otherwise
 *                TQ_DEVERR_SEQLEN_RANGE and the sequence gives 0.
 *   scale        softmax scale (typically 1/sqrt(D)).
 * K and V code widths (cb->k.bits, cb->v.bits): each of 2, 3, 4 and 8, in any pair
 * (TQ_ERR_UNSUPPORTED otherwise; tq_quantize_append takes 1..8).
 * H_q must be a multiple of H_kv with H_q / H_kv <= 16; block_size must be 16;
 * B * H_q < 2^31.  H_kv is at most 16 (8 when D = 256 or H_q / H_kv > 8), and a staged block of all
 * KV heads plus the code tables must fit in shared memory: with 8-bit tables that
 * excludes 16 KV heads at D = 128 and 8 at D = 256 (TQ_ERR_UNSUPPORTED;
 * tq_decode_plan_probe tells in advance).
 * One cooperative kernel launch: the merge of a sequence's partial results waits
 * (bounded, about 2 s) until every CTA that covers the sequence has published its
 * part; the merge work is spread over all CTAs.  A wait that gives up raises
 * TQ_DEVERR_TIMEOUT, leaves the affected query heads' output unwritten, and still
 * returns the merge counters to zero, so the next call runs normally.
 * Uses the per-device workspace (tq_set_workspace, or allocated by the library on
 * the first call that needs more, and kept until process exit).
 * Errors: TQ_ERR_INVALID_ARG / TQ_ERR_UNSUPPORTED / TQ_ERR_WORKSPACE (nothing
 * enqueued), TQ_ERR_CUDA. */
TQ_API tq_status tq_paged_decode(tq_tensor out, tq_tensor q, tq_tensor pages,
                          tq_tensor block_table, tq_tensor seq_lens,
                          const tq_codebooks* cb, uint64_t sign_seed, float scale,
                          void* stream);

/* The QJL residual sketch of the keys (tq-kv, "How It Works" step [5]: SRHT QJL error
 * correction; TorbuQuant, "Current Status": QJL residual).  After the Lloyd-Max code,
 * each K row also stores the 1-bit sketch of its rotated-domain residual r = u - c[idx]:
 * z_j = [(S r)_j >= 0] with S = (1/sqrt(D)) H diag(s2), a second randomized Hadamard
 * transform whose signs s2 come from SplitMix64 seeded with qjl_seed, and the fp32
 * gamma = ||r||.  K region = [packed codes | fp32 norm | D sign bits, LSB-first | fp32
 * gamma]; the V region follows unchanged.  Slot bytes: tq_slot_bytes_qjl (the pages'
 * slot_stride is at least that and a multiple of 8, so it may need padding).
 * Supported: D = 128 or 256 (the append), K widths 2, 3, 4 (the decode).  Same
 * arguments, layouts and errors as tq_quantize_append / tq_paged_decode otherwise; a
 * non-finite K row stores z = 0 and gamma = 0. */
TQ_API tq_status tq_slot_bytes_qjl(int32_t dim, int32_t k_bits, int32_t v_bits, int32_t* out);
TQ_API tq_status tq_quantize_append_qjl(tq_tensor pages, tq_tensor slot_mapping, tq_tensor k,
                                        tq_tensor v, const tq_codebooks* cb, uint64_t sign_seed,
                                        uint64_t qjl_seed, int32_t k_bits, int32_t v_bits,
                                        void* stream);
/* Decode over slots written by tq_quantize_append_qjl: each key is scored with its QJL
 * correction, scale nK (<R q, c[idx]> + gamma sqrt(pi/2)/sqrt(D) <S R q, 2z - 1>), the
 * second term as one more mma per k-step on +-1 fragments built from the sign bits. */
TQ_API tq_status tq_paged_decode_qjl(tq_tensor out, tq_tensor q, tq_tensor pages,
                                     tq_tensor block_table, tq_tensor seq_lens,
                                     const tq_codebooks* cb, uint64_t sign_seed,
                                     uint64_t qjl_seed, float scale, void* stream);

/* Paged decode with an uncompressed hot window (turboquant_pro 1.4.2, "Fused CUDA
 * decode": the fp16 hot window is merged through the online softmax, and "Streaming
 * cache"; tq-kv, "How It Works", "3-Fix for GGUF Models": sink tokens stay FP16, the
 * current token is lossless).  Same as tq_paged_decode, except that sequence b also
 * attends to hot tokens 0 .. hot_lens[b]-1 of hot_k / hot_v, inside the same softmax:
 *   out[b, h] = sum_t softmax_t(scale * <q[b,h], key_t>) value_t over the seq_lens[b]
 *               packed tokens (dequantized) and the hot tokens (read exactly).
 *   hot_k, hot_v  [B, W, H_kv, D] in bf16, f16 or f32 (same dtype and strides); the
 *                 last dim contiguous.  The caller keeps there whichever tokens stay
 *                 uncompressed (the first few "sink" tokens, the most recent ones); their
 *                 positions do not enter the result.  A token should be in the pages or
 *                 in the window, not both.
 *   hot_lens      i32 [B]; an entry outside [0, W] raises TQ_DEVERR_SEQLEN_RANGE and
 *                 counts as 0.  A sequence with seq_lens[b] == 0 attends to its hot
 *                 tokens alone; with no tokens at all it gives 0.
 * The packed tokens are reduced as in tq_paged_decode; the CTA that finishes a query
 * head computes the hot tokens' partial (fp32) and joins the two partials with one
 * rescale before the division by the softmax sum.
 * Errors: as tq_paged_decode, plus TQ_ERR_INVALID_ARG for mismatched hot tensors. */
TQ_API tq_status tq_paged_decode_hot(tq_tensor out, tq_tensor q, tq_tensor pages,
                                     tq_tensor block_table, tq_tensor seq_lens,
                                     tq_tensor hot_k, tq_tensor hot_v, tq_tensor hot_lens,
                                     const tq_codebooks* cb, uint64_t sign_seed, float scale,
                                     void* stream);

/* Allocation-free variant of tq_paged_decode (this library's own addition; the
 * pages describe no counterpart).  Same arguments, semantics and results as
 * tq_paged_decode, but its scratch is a fixed device array inside the library
 * (TQ_NOALLOC_SCRATCH_BYTES bytes, held by every device that loads the library
 * until the process exits) instead of a workspace the caller sets or the library
 * allocates.  It is meant for callers that must not allocate device memory on
 * the call path: a serving loop that keeps every allocation out of its steady
 * state (cudaMalloc/cudaFree can synchronise the device and fragment a pooled
 * allocator), or an embedding runtime that owns all device memory and forbids
 * libraries from allocating behind its back.  It calls no cudaMalloc, cudaFree or
 * allocating library routine.
 *
 *   - The first call on each device looks up the array's device address on that
 *     device (cudaGetSymbolAddress, which may load the library's module there);
 *     make that first call outside any stream capture.
 *   - A geometry whose scratch would exceed TQ_NOALLOC_SCRATCH_BYTES (see
 *     tq_decode_workspace_size for the size) is rejected with TQ_ERR_WORKSPACE and
 *     nothing is enqueued.
 *   - Every call on a device shares the one array.  It starts zeroed and every
 *     call leaves its merge counters at zero again.  Calls whose kernels overlap on
 *     the GPU (different streams without ordering) race on it: order them. */
#define TQ_NOALLOC_SCRATCH_BYTES (16u << 20)
TQ_API tq_status tq_paged_decode_noalloc(tq_tensor out, tq_tensor q, tq_tensor pages,
                                         tq_tensor block_table, tq_tensor seq_lens,
                                         const tq_codebooks* cb, uint64_t sign_seed, float scale,
                                         void* stream);

/* Attention of new tokens over the packed pages (this library's own addition next to
 * tq_paged_decode: the pages describe single-token decode only).  The new tokens' K and V
 * are already in the pages (tq_quantize_append first); sequence b's new tokens are the last
 * q_len[b] of its seq_lens[b], so the row of new token i of sequence b stands at position
 * p = seq_lens[b] - q_len[b] + i and attends to the tokens t <= p with
 *   window == 0  or  t > p - window  or  t < sinks
 * (causal; with window > 0 a sliding window plus the first `sinks` tokens):
 *   out[row, h] = sum_t softmax_t(scale * <q[row,h], k_hat_t>) v_hat_t, k_hat and v_hat as in
 *   tq_paged_decode.  A row that sees no token (p < 0, an empty sequence) gives 0.
 *   out, q       [rows, H_q, D] in bf16, f16 or f32 (out: f32 or q's dtype); last dim contiguous.
 *                Rows of q may overlap (a broadcast dim), those of out may not.
 *   q_starts     i32 [B + 1] contiguous, ascending: rows [q_starts[b], q_starts[b+1]) of q and
 *                out belong to sequence b.  Rows outside [q_starts[0], q_starts[B]) are neither
 *                read nor written.
 *   max_q        the largest q_len (host value; it sizes the grid).  A sequence with more new
 *                tokens, or a range that is not inside [0, rows], raises
 *                TQ_DEVERR_SEQLEN_RANGE and its rows are left unwritten.
 *   pages        u8 [num_blocks, 16, H_kv, slot_stride] as tq_quantize_append takes them:
 *                last dim contiguous, slot_stride >= tq_slot_bytes and a multiple of 8; block,
 *                row and head strides multiples of 8, data 8-byte aligned.
 *   block_table  i32 [B, max_blocks], last dim contiguous.  Entries of pages that no row sees
 *                are not read.  An entry outside [0, num_blocks) raises
 *                TQ_DEVERR_BLOCK_RANGE and its tokens are skipped.
 *   seq_lens     i32 [B]; outside [0, max_blocks * 16]: TQ_DEVERR_SEQLEN_RANGE, rows give 0.
 *   window, sinks  >= 0.
 * Code widths as in tq_paged_decode (each of 2, 3, 4, 8); D 64, 128 or 256; H_q a multiple of
 * H_kv; block_size 16; H_kv <= 65535, max_q * H_q / H_kv < 2^22, and B * H_kv * tiles of 8
 * query rows < 2^28 (TQ_ERR_UNSUPPORTED otherwise).
 * The operands of the two contractions are fp16, 8-bit key centroids twice that (hi + lo); sums
 * and softmax statistics are fp32.  Whatever the type of out, all rows together are within about
 * 1e-3 of the exact result in 2-norm (1,150 random calls: 1.4e-3 at most, in one of 8 rows; 2e-3
 * where a few keys have very large norms).  A single row may be further off: by 8e-3 of sum_t softmax_t |v_hat_t|, and
 * where its values cancel by 2e-2 of its own norm.  |q| is summed in fp32: below 1.8e19.
 * Only tokens a row sees reach its result: whatever the others' norms hold (a stored NaN or
 * infinite norm included).  out may be q itself.  No workspace, no state between calls: calls may
 * overlap on the GPU, and be captured (the library's first call on a device outside any capture).
 * The kernel and, without a window, how many blocks share a sequence's keys are chosen for the
 * whole call by max_q and block_table's width: give single tokens a call of their own next to long
 * chunks (2 chunks of 512 and 60 single tokens at 4,096: 553 us in one call, 123 + 121 in two), and
 * a table view no wider than the longest sequence (8 x 500 tokens in 32 columns 121 us, in 2,048
 * 203 us).
 * Errors: TQ_ERR_INVALID_ARG / TQ_ERR_UNSUPPORTED (nothing enqueued), TQ_ERR_CUDA. */
TQ_API tq_status tq_paged_attend(tq_tensor out, tq_tensor q, tq_tensor q_starts, tq_tensor pages,
                                 tq_tensor block_table, tq_tensor seq_lens,
                                 const tq_codebooks* cb, uint64_t sign_seed, float scale,
                                 int32_t max_q, int32_t window, int32_t sinks, void* stream);

/* The single-token form: tq_paged_attend with one new token a sequence (out, q [B, H_q, D]),
 * window > 0.  Reads the pages of the window and the sinks only, so that the others may have
 * been released (tq_pages_resize) and their entries be -1. */
TQ_API tq_status tq_paged_decode_window(tq_tensor out, tq_tensor q, tq_tensor pages,
                                        tq_tensor block_table, tq_tensor seq_lens,
                                        const tq_codebooks* cb, uint64_t sign_seed, float scale,
                                        int32_t window, int32_t sinks, void* stream);

/* Page operations (this library's own addition: the pages describe the page tensor and the
 * slot mapping, not who hands the pages out).  They keep the block table, the lengths and the
 * pages' reference counts of a batch on the device, so that a serving loop admits, extends,
 * forks, cuts and releases sequences without a host round trip.
 *   layers       host array of num_layers (1..128) page tensors, u8 [num_blocks, 16, H_kv,
 *                slot_stride] as in tq_paged_decode, all with the same num_blocks: the pools
 *                of a model's layers, which share one block table (H_kv and slot_stride may
 *                differ).  A page is contiguous; the stride between pages may be larger (a
 *                multiple of 16), so that several layers may interleave in one tensor.
 *                slot_stride a multiple of 8, data 16-byte aligned.
 *   block_table  i32 [B, max_blocks], last dim contiguous.  -1 marks an entry without a page.
 *   seq_lens     i32 [B] contiguous.
 *   ref_counts   i32 [num_blocks] contiguous: how many table entries name the page; 0 = free.
 *                The caller zeroes it once (and may count pages it keeps for itself).
 *   moves        i32 [requests, 2] contiguous, written by the call: {from, to} where the
 *                request got a copy of page `from` in page `to`, {-1, -1} where it needed
 *                none, {-2, -2} where it was refused.
 * Free pages are given out lowest index first, in the order of the requests.  A request
 * that, together with all requests before it, needs more pages than were free when the call
 * began is refused as a whole and leaves its sequence as it was (TQ_DEVERR_NO_PAGES); pages
 * released by a call are free for the next one.  Table entries outside [0, num_blocks) raise
 * TQ_DEVERR_BLOCK_RANGE where a count would change, and are skipped.
 * Calls that share tables, counts or pages must be ordered on the GPU.  No workspace; nothing
 * is allocated; every call can be captured (the library's first call on a device outside any
 * capture).
 * Limits (TQ_ERR_UNSUPPORTED): num_blocks <= 2^21, B and the number of pairs <= 8192,
 * max_blocks < 2^26.
 * Errors: TQ_ERR_INVALID_ARG / TQ_ERR_UNSUPPORTED (nothing enqueued), TQ_ERR_CUDA. */

/* Every sequence b gets new_lens[b] tokens (i32 [B]; equal to seq_lens[b]: unchanged; 0: the
 * sequence is released), and seq_lens[b] = new_lens[b].
 *   growing    new entries name free pages.  If the sequence's last page is partly filled and
 *              shared (count > 1), it is first replaced by a copy of its own, in every layer.
 *   shrinking  the entries past the new length are released and set to -1.  (A
 *              sequence cut back into pages that a window released keeps their -1 entries.)
 *   window > 0 entries of pages that no query at position min(old, new length) or later can
 *              see through a sliding window with sinks (tq_paged_attend) are released too and
 *              set to -1.  The window kernels never read such entries.  0: none.
 * A length outside [0, max_blocks * 16] raises TQ_DEVERR_SEQLEN_RANGE and leaves the sequence
 * as it is (moves {-2, -2}).  moves: [B, 2]. */
TQ_API tq_status tq_pages_resize(const tq_tensor* layers, int32_t num_layers, tq_tensor block_table,
                                 tq_tensor seq_lens, tq_tensor new_lens, tq_tensor ref_counts,
                                 tq_tensor moves, int32_t window, int32_t sinks, void* stream);

/* Sequence children[i] becomes a copy of sequence parents[i] (i32 [N] each): it shares the
 * parent's full pages (their counts go up) and gets its own copy of a partly filled last
 * page, so that both may append.  Lengths are those at the start of the call.  A child must be
 * empty (seq_lens 0) and named once; otherwise, or for an index outside [0, B), the pair is
 * refused with TQ_DEVERR_SEQ_INDEX.  moves: [N, 2]. */
TQ_API tq_status tq_pages_fork(const tq_tensor* layers, int32_t num_layers, tq_tensor block_table,
                               tq_tensor seq_lens, tq_tensor ref_counts, tq_tensor parents,
                               tq_tensor children, tq_tensor moves, void* stream);

/* Gathers kept tokens: token i < counts[b] of sequence b in the pages of dst_table becomes a
 * copy of its token positions[b, i] in the pages of src_table, in every layer (K and V slots
 * of all heads).  Any order and repetition; kept tokens in ascending order compact a cache
 * after eviction, all tokens copy or move a sequence.
 *   src_table   i32 [B, max_blocks], src_lens i32 [B].
 *   positions   i32 [B, P], last dim contiguous; counts i32 [B] contiguous.
 *   dst_table   i32 [B, dst_blocks] (from tq_pages_resize on the destination's tables).
 * Only rows [0, counts[b]) are written: the rest of the last page stays.  No destination page
 * may be read by the same call or written twice (its bytes would be unspecified).
 * A count outside [0, min(P, dst_blocks * 16)] or a source length outside the table raises
 * TQ_DEVERR_SEQLEN_RANGE and skips the sequence; a position outside [0, src_lens[b]) raises
 * TQ_DEVERR_SLOT_RANGE, a table entry outside [0, num_blocks) TQ_DEVERR_BLOCK_RANGE, and the
 * row is skipped.  Lengths and counts are left to the caller. */
TQ_API tq_status tq_pages_compact(const tq_tensor* layers, int32_t num_layers, tq_tensor src_table,
                                  tq_tensor src_lens, tq_tensor positions, tq_tensor counts,
                                  tq_tensor dst_table, void* stream);

/* Workspace bytes tq_paged_decode needs for this geometry (host only).  The
 * workspace holds 2 * batch u32 merge counters at its start (zero between calls:
 * each call clears the ones it raised) and the split-KV partial results (m, l, O')
 * in fp32. */
TQ_API tq_status tq_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t max_blocks, int32_t block_size,
                                   size_t* bytes);

/* Give the library a caller-owned device workspace for the CURRENT device
 * (ptr 256-byte aligned; NULL releases the association).  The library zeroes it
 * here (cudaMemset, synchronous) and never frees it; the caller must not write to
 * it while it is set.  Calls that use one device's workspace must be ordered on the
 * GPU (one stream, or events); concurrent decodes on one device race on it. */
TQ_API tq_status tq_set_workspace(void* ptr, size_t bytes);

/* Read and clear the current device's error word (TQ_DEVERR_* bits).  Host
 * pointer `out`; synchronises `stream` first.  When the word is non-zero it also
 * clears the merge counters of the device's workspaces, which a failed decode may
 * have left raised. */
TQ_API tq_status tq_get_device_error(int32_t* out, void* stream);

/* Test export of the rotation used by tq_quantize_append: for each row x of
 * `x` [N, D] (bf16/f16/f32), writes u = y / n with y = (1/sqrt(D)) H (s*x), n = ||x||,
 * in fp32 to `u` [N, D] and fp32(n) to `norm` [N], computed with exactly the
 * device arithmetic the append kernel uses (so encoding these u on the host
 * reproduces the kernel's codes bit for bit). */
TQ_API tq_status tq_rotate_unit(tq_tensor u, tq_tensor norm, tq_tensor x, uint64_t sign_seed,
                         void* stream);

/* Quantize-append with the dense rotation (turboquant_serve 0.1.2, "Architecture":
 * rotate k, v = k @ R, then normalize, encode and pack; turboquant_pro 1.4.2, "Fused CUDA
 * decode": rotation and quantization in one tiled GEMM).  Same slot layout, norm,
 * encode and errors as tq_quantize_append, with y = R x in place of the randomized
 * Hadamard transform: u = y / ||x||.  y is one tcgen05 GEMM per tile of 128 (token, head)
 * rows (bf16 x bf16 -> fp32 in tensor memory, R as hi and lo).
 *   rot   host pointer; rot->dim == D.
 * Supported: D = 64 or 128; k, v bf16, 16-byte aligned with token and head strides that
 * are multiples of 8 elements; H_kv a divisor or a multiple of 128 (TQ_ERR_UNSUPPORTED
 * otherwise).  Rows whose sum of squares leaves [2^-60, 2^100] are rotated on the CUDA
 * cores after an exact power-of-two rescaling. */
TQ_API tq_status tq_quantize_append_dense(tq_tensor pages, tq_tensor slot_mapping, tq_tensor k,
                                          tq_tensor v, const tq_codebooks* cb,
                                          const tq_rotation* rot, int32_t k_bits, int32_t v_bits,
                                          void* stream);

/* Paged decode with the dense rotation: as tq_paged_decode (sign_seed unused), with
 * q' = R q and o = R^T O' / l (fp32 on the CUDA cores, once per query head). */
TQ_API tq_status tq_paged_decode_dense(tq_tensor out, tq_tensor q, tq_tensor pages,
                                       tq_tensor block_table, tq_tensor seq_lens,
                                       const tq_codebooks* cb, const tq_rotation* rot, float scale,
                                       void* stream);

/* Test export of the dense append's rotation: for each bf16 row x of `x` [N, D] writes
 * u = R x / ||x|| (fp32, [N, D], unit stride) and fp32(||x||) to `norm` [N] with exactly
 * the arithmetic of tq_quantize_append_dense (the same kernel), so that encoding these u
 * on the host reproduces its codes bit for bit.  Same limits as that call. */
TQ_API tq_status tq_rotate_unit_dense(tq_tensor u, tq_tensor norm, tq_tensor x,
                                      const tq_rotation* rot, void* stream);

/* Test export for failure detection without a GPU fault (this library's own addition;
 * the pages describe no counterpart).  The NEXT decode launch on the current device
 * (tq_paged_decode or tq_paged_decode_noalloc) bounds its waits by `wait_ms`
 * milliseconds instead of about 2 s, and its CTA number `withhold_cta` never announces
 * its partial results.  So the CTAs that share a sequence with it give up waiting, raise
 * TQ_DEVERR_TIMEOUT, and write no output for that sequence (a withheld CTA past the
 * grid changes nothing).  One shot: later launches are normal.  Host only; nothing is
 * enqueued.
 * Errors: TQ_ERR_INVALID_ARG for withhold_cta < 0 or wait_ms outside 1..2000. */
TQ_API tq_status tq_debug_inject_merge_stall(int32_t withhold_cta, int32_t wait_ms);

/* Test export of the decode kernel's shared-memory plan for one call geometry on a
 * device described by num_sms, max_smem_optin (bytes one CTA may use) and
 * dyn_smem_base (the shared-window address where dynamic shared memory starts).
 * Host only: no device call.  out[14] receives, in order: wph, nst, row_pitch,
 * stage_bytes, lut_win, lut_off, lut_bytes, stage_lo_off, stage_hi_off, n_low,
 * misc_off, smem bytes, copy_mode (1: 2-D tensor box, 0: 1-D bulk copy), warps per CTA.
 * Errors: TQ_ERR_INVALID_ARG for out == NULL or non-positive sizes; TQ_ERR_UNSUPPORTED
 * when no layout fits. */
TQ_API tq_status tq_decode_plan_probe(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t head_dim, int32_t k_bits, int32_t v_bits,
                                      int32_t slot_stride, int32_t max_blocks, int32_t num_sms,
                                      int32_t max_smem_optin, uint32_t dyn_smem_base,
                                      int64_t* out);

/* Static description of a status code (never NULL). */
TQ_API const char* tq_status_string(tq_status status);

/* Library version, e.g. "0.1.0". */
TQ_API const char* tq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TQ_H_ */
