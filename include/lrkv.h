/*
 * lrkv.h -- C ABI of the GB300 (sm_103a) library for attention over an
 * LRKV-compressed KV cache.
 *
 * The method ("Low-Rank Key Value Attention", O'Neill, Clancy, Matskevichus,
 * Reid, arXiv:2601.11471v3; slide deck of the same title):
 *   each head's key/value projection is W_h = W_shared + U_h B_h^T
 *   (Eqs. (2)-(3), frame "LRKV constrains differences between heads"), so per
 *   token and layer the cache holds a shared d_h-vector s plus one r-vector z_h
 *   per head, for keys and for values: 2(d_h + H r) elements (frame "Can heads
 *   share storage while keeping distinct K/V features?").  Decode never expands
 *   per-head keys or values; it evaluates the factored forms of Eqs. (6)-(7).
 *
 * Conventions shared by every entry point
 *   - All tensors are bf16 (IEEE binary16 brain-float bit patterns, uint16 in
 *     memory) unless stated, row-major, in DEVICE memory owned by the caller.
 *     The library allocates nothing and keeps no state between calls.
 *   - Every pointer must be 16-byte aligned.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *     asynchronous: they validate on the host, enqueue kernels and return.
 *   - Host-detectable errors are returned before anything is launched; the
 *     calling thread can then read a one-line explanation from
 *     lrkv_last_error().  A launch failure returns LRKV_ERR_CUDA.
 *   - Errors only the device can see (an index read from device memory that is
 *     out of range, a bounded wait that expired) are OR-ed into the optional
 *     uint32 word `status_dev` (device memory, may be NULL) as LRKV_DEV_* bits;
 *     the offending access is skipped, never trapped.  Read the word after
 *     synchronising the stream.
 *   - Cache pages: the pools are indexed by physical block id b in
 *     [0, num_blocks); token slot = b * block_size + offset.
 *        sK     : [num_blocks][block_size][d_h + d_rope]   rows [s^K | k^R]
 *        sV     : [num_blocks][block_size][d_h]
 *        zK, zV : [num_blocks][block_size][H][r]
 *     (s = shared features K_s, V_s of Eq. (4); z_h = per-head latents R_h^K,
 *     R_h^V of Eq. (5); k^R = the optional decoupled positional key, below.)
 *     B_h^K, B_h^V are weights, not cache entries.
 *   - Decoupled positional key (d_rope > 0; "Low-Rank Key Value Attention",
 *     combination with MLA-style latent caches, whose decoupled rotary key is
 *     one d_rope-vector per token shared by all heads): every key row carries
 *     k^R = RoPE(x W^KR, pos) after s^K.  A query is then [q | q^R] (q^R already
 *     rotated by the caller), logits are q . (s^K + B_h^K z^K_h) + q^R . k^R, and
 *     the default scale is 1/sqrt(d_h + d_rope).  RoPE turns the pair (2i, 2i+1)
 *     of a d_rope-vector by the angle pos * rope_base^(-2i / d_rope).  Values
 *     carry no positional part.  d_rope == 0 is the plain method, bit for bit.
 *
 * Supported shapes (others return LRKV_ERR_UNSUPPORTED):
 *   block_size == 64, d_h in {64, 128}, r in {8, 16, 32} with r <= d_h,
 *   1 <= H <= 128, d a positive multiple of 8 (of 64 for the tensor-core append),
 *   d_rope in {0, 64}.  The decode calls with r = 32 and H >= 105 need H a multiple
 *   of 8: a stage of the scan then holds the latents of a group of heads, not of all.
 */
#ifndef LRKV_H
#define LRKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* 3: lrkv_dims.num_splits and the layer-batched calls; 4: lrkv_prefill_fused,
 * lrkv_decode_partials and lrkv_decode_merge (no struct changed). */
#define LRKV_ABI_VERSION 4

typedef enum lrkv_status {
    LRKV_OK = 0,
    LRKV_ERR_INVALID_ARG = 1,   /* NULL or misaligned pointer, negative size, inconsistent arguments */
    LRKV_ERR_UNSUPPORTED = 2,   /* shape outside the supported set above */
    LRKV_ERR_WORKSPACE = 3,     /* workspace smaller than the *_workspace_bytes() figure */
    LRKV_ERR_CUDA = 4,          /* a CUDA runtime call or kernel launch failed */
    LRKV_ERR_DEVICE_BOUNDS = 5, /* meaning of the LRKV_DEV_BAD_* bits, for lrkv_status_string */
    LRKV_ERR_TIMEOUT = 6        /* meaning of the LRKV_DEV_TIMEOUT bit, for lrkv_status_string */
} lrkv_status;

/* Bits kernels OR into *status_dev. */
#define LRKV_DEV_BAD_BLOCK 0x1u  /* a block_table entry needed by a call is outside [0, num_blocks) */
#define LRKV_DEV_BAD_SEQLEN 0x2u /* seq_len / q_start + Tq outside [1, max_blocks_per_seq * block_size]; that
                                    sequence's output rows are written as zeros */
#define LRKV_DEV_BAD_SLOT 0x4u   /* slot_mapping entry >= num_blocks * block_size (row skipped) */
#define LRKV_DEV_TIMEOUT 0x8u    /* a pipeline wait in a kernel gave up after its time limit (about 2 s) */
#define LRKV_DEV_NO_PAGES 0x10u  /* a sequence asked for more pages than are free and got none */
#define LRKV_DEV_BAD_INDEX 0x20u /* an index of a sequence or drafted token is out of range, out of order or listed
                                    twice, or a page with reference count 0 was given back */

/* Model dimensions (frame "LRKV constrains differences between heads"). */
typedef struct lrkv_dims {
    int32_t H;           /* query heads */
    int32_t d_h;         /* head width */
    int32_t r;           /* residual rank of U_h B_h^T */
    int32_t d;           /* hidden size of the rows appended to the cache */
    int32_t block_size;  /* tokens per cache page; must be 64 */
    float softmax_scale; /* logit scale; 0 means 1/sqrt(d_h + d_rope) (frame "Compute logits ...") */
    int32_t d_rope;      /* width of the decoupled positional key shared by all heads; 0 = none */
    float rope_base;     /* RoPE base; 0 means 10000 (ignored when d_rope == 0) */
    int32_t num_splits;  /* decode only: how many equal contiguous pieces the batch's cached tokens
                            are cut into for the split-K scan (each piece is scanned by one CTA and
                            leaves one partial softmax state per sequence it touches); 0 = one per
                            SM (the default), else 1..65536.  Results agree across values up to
                            floating-point rounding. */
} lrkv_dims;

/* One layer's paged cache (device pointers, caller-owned, layout above). */
typedef struct lrkv_cache {
    void* sK;
    void* sV;
    void* zK;
    void* zV;
    int32_t num_blocks;
} lrkv_cache;

/* ABI version of the loaded library (LRKV_ABI_VERSION it was built with). */
int lrkv_abi_version(void);

/* Static description of a status code. */
const char* lrkv_status_string(lrkv_status s);

/* Explanation of the last non-OK status returned on the calling thread ("" if none). */
const char* lrkv_last_error(void);

/* Bytes of one cache page across the four pools: block_size * 2 * (2(d_h + H r) + d_rope).
 * Returns 0 for unsupported dims. */
size_t lrkv_cache_block_bytes(const lrkv_dims* dims);

/*
 * lrkv_append -- Eqs. (4)-(5): project n_tok hidden rows into the cache.
 *   Y = X W_cat, W_cat = [W_shared^K | W^KR | W_shared^V | U_1^K .. U_H^K | U_1^V .. U_H^V]
 *   (d x N, N = 2(d_h + H r) + d_rope; W^KR absent when d_rope == 0), accumulated
 *   in fp32; the d_rope columns of W^KR are then rotated at positions[t] (angle in
 *   double, sine and cosine in fp32 corrected to first order in double, products in
 *   double, result rounded to fp32: within ~1e-7 of the pair's magnitude of the exact
 *   rotation); everything is rounded to bf16
 *   (nearest, ties to even).  Row t is written to token slot slot_mapping[t]:
 *   columns [0, d_h + d_rope) -> sK, the next d_h -> sV, the next H r -> zK
 *   (head-major), the last H r -> zV.
 *   X            [n_tok][d]
 *   W_catT       [N][d]  (W_cat transposed: row c holds the weights of output column c)
 *   slot_mapping [n_tok] int32 (device); a negative entry skips the row,
 *                an entry >= num_blocks*block_size sets LRKV_DEV_BAD_SLOT and skips it.
 *   positions    [n_tok] int32 (device) token positions, >= 0; required when
 *                d_rope > 0, ignored (may be NULL) otherwise.
 *   n_tok == 0 is a no-op.  Small n_tok runs a bandwidth-bound kernel, large n_tok a
 *   tcgen05 tensor-core GEMM; both give bit-identical results whenever every fp32
 *   partial sum is exact.
 */
lrkv_status lrkv_append(const lrkv_dims* dims, const void* X, const void* W_catT, int32_t n_tok,
                        const int32_t* slot_mapping, const int32_t* positions, const lrkv_cache* cache,
                        uint32_t* status_dev, void* stream);

/* Workspace bytes lrkv_decode needs for `batch` sequences on the CURRENT device (for
 * lrkv_decode_layers pass num_layers * batch). */
size_t lrkv_decode_workspace_bytes(const lrkv_dims* dims, int32_t batch);

/*
 * lrkv_decode -- one decode step per sequence, factored form (Eqs. (6)-(7)):
 *   q~_h = q_h B_h^K;  score_t = (q_h . s^K_t + q~_h . z^K_{h,t}) * scale;
 *   a_h = softmax_t(score);  out_h = a_h V_s + (a_h R_h^V) (B_h^V)^T.
 *   The query attends to all seq_lens[b] cached tokens (positions 0..L-1; it is
 *   the newest position and is already in the cache).  Split over the sequence
 *   across the GPU's SMs, merged by log-sum-exp in a second kernel.  With a
 *   positional key the logit gains q^R . k^R_t (see the conventions above).
 *   q           [batch][H][d_h + d_rope]  ([q_h | q^R_h]; q~ uses the first d_h)
 *   BK, BV      [H][d_h][r]  (B_h^K, B_h^V)
 *   block_table [batch][max_blocks_per_seq] int32 (device)
 *   seq_lens    [batch] int32 (device)
 *   out         [batch][H][d_h]
 *   workspace   device scratch of >= lrkv_decode_workspace_bytes(dims, batch) bytes, 256-byte aligned.
 *   Capacity of one call: batch x max_blocks_per_seq x block_size below 2^34 tokens (times
 *   num_layers for lrkv_decode_layers); larger calls return LRKV_ERR_INVALID_ARG.
 */
lrkv_status lrkv_decode(const lrkv_dims* dims, const void* q, const void* BK, const void* BV,
                        const lrkv_cache* cache, const int32_t* block_table, int32_t max_blocks_per_seq,
                        const int32_t* seq_lens, int32_t batch, void* out, void* workspace,
                        size_t workspace_bytes, uint32_t* status_dev, void* stream);

/*
 * lrkv_decode_fused -- lrkv_decode with both absorptions moved into the caller's
 *   weights (the associativity of frame "Compute logits without expanding
 *   historical keys", step 1, and of Eq. (7), "reduce the latents to one r-vector,
 *   then map"): the query arrives with q~_h = x (W_h^Q B_h^K) already projected,
 *   and the output is returned before the residual up-projection, for an output
 *   projection with B_h^V folded into W^O.  Per sequence b and head h:
 *     score_t = ([q_h | q~_h] . [s^K_t | z^K_{h,t}]) * scale;  a_h = softmax_t(score)
 *     out_h   = [ sum_t a_t s^V_t  |  sum_t a_t z^V_{h,t} ]        (width d_h + r)
 *   i.e. single-head softmax attention over the concatenated features (with a
 *   positional key, [q_h | q^R_h | q~_h] . [s^K_t | k^R_t | z^K_{h,t}]).
 *   q           [batch][H][d_h + d_rope]   bf16
 *   q_tilde     [batch][H][r]     bf16, 16-byte aligned
 *   out         [batch][H][d_h + r] bf16 (nearest, ties to even from fp32)
 *   Everything else (cache, block_table, seq_lens, workspace, status, errors, the
 *   stream) is as for lrkv_decode; no B^K or B^V is read.  Unlike lrkv_decode, the
 *   call does not overlap the caller's previous kernel on the stream.
 */
lrkv_status lrkv_decode_fused(const lrkv_dims* dims, const void* q, const void* q_tilde, const lrkv_cache* cache,
                              const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                              int32_t batch, void* out, void* workspace, size_t workspace_bytes,
                              uint32_t* status_dev, void* stream);

/*
 * lrkv_decode_partials / lrkv_decode_merge -- lrkv_decode cut at the log-sum-exp merge, for a
 *   sequence whose cached tokens are spread over several caches (e.g. one token range per
 *   device).  The online softmax of frame "Compute logits without expanding historical keys"
 *   is associative over any split of the tokens, and B_h^V is applied after the merge (Eq. (7):
 *   the latents are aggregated first), so each part only has to return, per (sequence, head),
 *   over its own tokens t:
 *     m   = max_t s_t,  s_t = ([q | q~] . [s^K_t | z^K_{h,t}]) * scale * log2(e)
 *     l   = sum_t 2^(s_t - m)
 *     acc = sum_t 2^(s_t - m) [s^V_t | z^V_{h,t}]                    (width d_h + r)
 *   and the merge of P parts is M = max_p m_p, w_p = 2^(m_p - M),
 *     out_h = (sum_p w_p acc_s,p + B_h^V sum_p w_p acc_z,p) / sum_p w_p l_p.
 *   lrkv_decode_partials: arguments as lrkv_decode (no B^V, no out); seq_lens[b] counts the
 *     tokens of sequence b held in THIS cache and may be 0 (an empty part: m = -inf, l = 0,
 *     acc = 0; no status bit).
 *     partials  [batch][H][d_h + r + 2] fp32: acc_s (d_h), acc_z (r), m, l
 *   lrkv_decode_merge: partials [num_parts][batch][H][d_h + r + 2] (the parts' outputs stacked,
 *     e.g. by an all-gather), BV as for lrkv_decode, out [batch][H][d_h] bf16 (nearest, ties to
 *     even).  A (sequence, head) that no part holds a token of gets zeros and
 *     LRKV_DEV_BAD_SEQLEN.  num_parts >= 1; 1 <= batch <= 65535 (0 is a no-op).
 *   Pointers 16-byte aligned, device memory, the caller's stream; errors as for lrkv_decode.
 */
lrkv_status lrkv_decode_partials(const lrkv_dims* dims, const void* q, const void* BK, const lrkv_cache* cache,
                                 const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                 int32_t batch, float* partials, void* workspace, size_t workspace_bytes,
                                 uint32_t* status_dev, void* stream);
lrkv_status lrkv_decode_merge(const lrkv_dims* dims, int32_t num_parts, const float* partials, const void* BV,
                              int32_t batch, void* out, uint32_t* status_dev, void* stream);

/*
 * lrkv_decode_static_ws -- lrkv_decode without a caller workspace.  (The paper has
 *   no counterpart; this is a deployment convenience.)
 *   For callers that cannot allocate device memory: cudaMalloc/cudaFree can
 *   synchronise the whole device and stall other streams, some host frameworks
 *   own the GPU allocator and forbid foreign allocations, and some deployments fix
 *   their device-memory budget at start-up.  The scratch lives in a fixed array of
 *   LRKV_STATIC_WS_BYTES inside the library's device image, which every GPU that
 *   loads the library keeps until the process exits; this call allocates nothing.
 *   Arguments, layouts and results are those of lrkv_decode.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.  The address is kept per device together with
 *     the id of the context it was found in; after a device reset (a new context,
 *     which loads the library's device image afresh) the next call looks it up
 *     again, so make that call outside a stream capture too.
 *   - Returns LRKV_ERR_WORKSPACE (explained by lrkv_last_error()) when
 *     lrkv_decode_workspace_bytes(dims, batch) exceeds LRKV_STATIC_WS_BYTES.
 *   - All calls on a device share the one array, which keeps the last call's
 *     contents (nothing needs clearing: each call writes all scratch it reads).
 *     Calls whose kernels overlap on the GPU -- e.g. on two streams at once --
 *     race on it; serialise them.
 */
#define LRKV_STATIC_WS_BYTES ((size_t)16 << 20)
lrkv_status lrkv_decode_static_ws(const lrkv_dims* dims, const void* q, const void* BK, const void* BV,
                                  const lrkv_cache* cache, const int32_t* block_table, int32_t max_blocks_per_seq,
                                  const int32_t* seq_lens, int32_t batch, void* out, uint32_t* status_dev,
                                  void* stream);

/* ======================================================================
 * Layer-batched calls: one launch of each kernel for several layers.
 *
 * A decode step of an L-layer model appends one row per sequence and attends over every
 * layer's cache.  Each layer has its own weights, cache pools, queries and outputs; the block
 * table and the lengths are the same for all layers.  When the queries of several layers are
 * known together (independent layers, or layers whose inputs are already computed), these
 * calls do the work of num_layers calls of lrkv_append / lrkv_decode in one launch per kernel,
 * with the whole batch's cached tokens of all layers divided evenly over the SMs -- many small
 * layers otherwise pay each kernel's fixed start-up and drain cost once per layer.
 *
 * Layer l's tensor is found at (layer 0's pointer) + l * stride, strides in bf16 elements
 * (multiples of 8, so every layer's tensors stay 16-byte aligned, and at least the size of
 * one layer's tensor: layers do not overlap).  The `cache` argument holds layer 0's pools
 * and num_blocks, the number of blocks of each layer's pools.
 * ====================================================================== */
typedef struct lrkv_layer_strides {
    int64_t X, W_catT;      /* lrkv_append_layers: hidden rows [n_tok][d], W_cat^T [N][d] */
    int64_t q, BK, BV, out; /* lrkv_decode_layers: [batch][H][d_h + d_rope], [H][d_h][r] (x2), [batch][H][d_h] */
    int64_t sK, sV, zK, zV; /* cache pools of both calls */
} lrkv_layer_strides;

/*
 * lrkv_append_layers -- lrkv_append of the same n_tok token slots (slot_mapping, positions)
 *   in num_layers layers: layer l's rows X_l W_cat,l go to layer l's pools.  Everything else
 *   as for lrkv_append; num_layers == 1 is lrkv_append (strides ignored, may be NULL).
 */
lrkv_status lrkv_append_layers(const lrkv_dims* dims, int32_t num_layers, const lrkv_layer_strides* strides,
                               const void* X, const void* W_catT, int32_t n_tok, const int32_t* slot_mapping,
                               const int32_t* positions, const lrkv_cache* cache, uint32_t* status_dev,
                               void* stream);

/*
 * lrkv_decode_layers -- lrkv_decode of the same batch (block_table, seq_lens) in num_layers
 *   layers: out_l = decode(q_l, B^K_l, B^V_l, cache_l), Eqs. (6)-(7) per layer.  The workspace
 *   is lrkv_decode_workspace_bytes(dims, num_layers * batch) bytes.  Everything else as for
 *   lrkv_decode; num_layers == 1 is lrkv_decode (strides ignored, may be NULL).
 */
lrkv_status lrkv_decode_layers(const lrkv_dims* dims, int32_t num_layers, const lrkv_layer_strides* strides,
                               const void* q, const void* BK, const void* BV, const lrkv_cache* cache,
                               const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                               int32_t batch, void* out, void* workspace, size_t workspace_bytes,
                               uint32_t* status_dev, void* stream);

/* ======================================================================
 * Quantised cache: the same pages with 8 bits a value.
 *
 * A token's row holds its four parts s^K (d_h + d_rope values), s^V (d_h), z^K (H r) and z^V (H r)
 * in blocks of 32 consecutive values (a part's last block may be shorter), each with one scale
 * 2^k.  With amax the block's largest magnitude,
 *     k = floor(log2 amax) - 6 (at least -126),   q_i = min(127, max(-127, rint(x_i / 2^k)))
 * (rint: nearest, ties to even), so |x_i - q_i 2^k| <= 2^(k-1) <= 2^-7 amax for amax >= 2^-120, and
 * q_i 2^k is exact in bf16.  A block that holds a NaN or an infinity reads as NaN throughout.
 *   row : [s^K | s^V | z^K, padded to 16 | z^V, padded to 16 | scales of s^K, s^V, z^K, z^V], bytes;
 *         a value's byte is q_i + 128, a block's scale byte k + 127 (255: NaN block; 0: zeros, as
 *         in memory that was cleared); padded to an odd number of 16-byte units
 *   rows: [num_blocks][block_size][lrkv_quant_row_bytes()]
 * The row is 1.03 bytes a value instead of 2.  Block tables, slots and lengths are as for the
 * bf16 pools; the same dims as for lrkv_decode are supported (r = 32 with any H).
 * ====================================================================== */
typedef struct lrkv_quant_cache {
    void* rows;          /* device pointer, 16-byte aligned */
    int32_t num_blocks;
} lrkv_quant_cache;

/* Bytes of one token's row, and of one page (block_size rows); 0 for unsupported dims. */
size_t lrkv_quant_row_bytes(const lrkv_dims* dims);
size_t lrkv_quant_block_bytes(const lrkv_dims* dims);

/*
 * lrkv_cache_quantize -- write n_tok rows of a quantised cache from rows of bf16 pools (those a
 *   lrkv_append has just written, or whole pages that move to 8 bits).
 * lrkv_cache_dequantize -- read n_tok rows back into bf16 pools (exactly: no rounding).
 *   Row i is moved between token slot bf16_slots[i] of `cache` and token slot quant_slots[i] of
 *   `qcache`.
 *   bf16_slots, quant_slots [n_tok] int32 (device); where either is negative the row is skipped;
 *     one at or beyond its cache's num_blocks * block_size sets LRKV_DEV_BAD_SLOT and skips it.
 *     The slots written by a call must differ from one another: of two rows written to one slot
 *     any mixture may remain.
 *   Slots that are not named keep their contents.  n_tok == 0 is a no-op.
 */
lrkv_status lrkv_cache_quantize(const lrkv_dims* dims, int32_t n_tok, const lrkv_cache* cache,
                                const int32_t* bf16_slots, const lrkv_quant_cache* qcache,
                                const int32_t* quant_slots, uint32_t* status_dev, void* stream);
lrkv_status lrkv_cache_dequantize(const lrkv_dims* dims, int32_t n_tok, const lrkv_quant_cache* qcache,
                                  const int32_t* quant_slots, const lrkv_cache* cache, const int32_t* bf16_slots,
                                  uint32_t* status_dev, void* stream);

/* Workspace bytes of the two decode calls below for `batch` sequences on the CURRENT device. */
size_t lrkv_decode_quant_workspace_bytes(const lrkv_dims* dims, int32_t batch);

/*
 * lrkv_decode_quant -- lrkv_decode over a quantised cache: the same formulas on the values q_i 2^k
 *   that the rows stand for, read as they are (nothing is dequantised into memory).
 * lrkv_decode_quant_partials -- its lrkv_decode_partials: per (sequence, head) the unnormalised
 *   state over this cache's tokens, for lrkv_decode_merge (e.g. old tokens here, the newest ones
 *   or a shared prefix in bf16 pools).
 *   Arguments, lengths, errors and status bits are those of lrkv_decode / lrkv_decode_partials with
 *   `qcache` in place of the pools; workspace of lrkv_decode_quant_workspace_bytes(dims, batch)
 *   bytes, 256-byte aligned.  All sums are fp32.  The products take q and q~ in fp16, each head's q and each
 *   head's q~ divided by a power of two of its own, that of its largest magnitude: 11 significant bits down to 2^-14
 *   of the largest, half a step of 2^-25 of it below.  Probabilities enter the products with s^V in bf16 and those
 *   with z^V in fp16 (times the tokens' scales, relative to the largest such weight).
 */
lrkv_status lrkv_decode_quant(const lrkv_dims* dims, const void* q, const void* BK, const void* BV,
                              const lrkv_quant_cache* qcache, const int32_t* block_table, int32_t max_blocks_per_seq,
                              const int32_t* seq_lens, int32_t batch, void* out, void* workspace,
                              size_t workspace_bytes, uint32_t* status_dev, void* stream);
lrkv_status lrkv_decode_quant_partials(const lrkv_dims* dims, const void* q, const void* BK,
                                       const lrkv_quant_cache* qcache, const int32_t* block_table,
                                       int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch,
                                       float* partials, void* workspace, size_t workspace_bytes,
                                       uint32_t* status_dev, void* stream);

/* ======================================================================
 * Shared prefix: one decode step of a batch whose sequences begin with the same tokens.
 *
 * The prefix's rows sit once in the cache, in pages listed by prefix_blocks; each sequence goes on
 * in pages of its own (block_table, seq_lens, as for lrkv_decode; a length may be 0).  Softmax
 * attention over both is the log-sum-exp merge of the two parts' states, so the prefix is read
 * once for all sequences, whose queries share its products on the tensor cores.
 * ====================================================================== */

/* Workspace bytes of the two calls below for `batch` sequences and prefixes of up to
 * max_prefix_blocks pages, on the CURRENT device. */
size_t lrkv_decode_shared_workspace_bytes(const lrkv_dims* dims, int32_t batch, int32_t max_prefix_blocks);

/*
 * lrkv_decode_shared -- out_h = softmax attention (Eqs. (6)-(7)) over the prefix_len[0] tokens of the
 *   prefix followed by the sequence's own seq_lens[b] tokens.
 *   prefix_blocks [max_prefix_blocks] int32 (device) pages of the prefix, in order
 *   prefix_len    [1] int32 (device), in [0, max_prefix_blocks * block_size]; 0: no prefix
 *   Everything else as for lrkv_decode, except that seq_lens[b] may be 0.  A prefix_len or length
 *   outside its range, or no token at all, sets LRKV_DEV_BAD_SEQLEN and writes zeros (a bad
 *   prefix_len: for all sequences).  A page id of the prefix outside [0, num_blocks) sets
 *   LRKV_DEV_BAD_BLOCK and its tokens are left out.  Rows behind the prefix's last token may hold
 *   any bits.  A NaN or infinity in a head's latents stays in that head, as in lrkv_decode (a page
 *   that holds one takes longer).  The
 *   prefix's products take the probabilities in bf16 and q~ in two bf16 pieces and sum in fp32.
 *   The work is planned from the tables' widths (the lengths are on the device): max_prefix_blocks and
 *   max_blocks_per_seq well above what is in use are allowed, but cost time.
 * lrkv_prefix_partials -- the prefix's part alone, as lrkv_decode_partials returns it (for
 *   lrkv_decode_merge with the partials of other caches); prefix_len 0 gives empty partials.
 */
lrkv_status lrkv_decode_shared(const lrkv_dims* dims, const void* q, const void* BK, const void* BV,
                               const lrkv_cache* cache, const int32_t* prefix_blocks, int32_t max_prefix_blocks,
                               const int32_t* prefix_len, const int32_t* block_table, int32_t max_blocks_per_seq,
                               const int32_t* seq_lens, int32_t batch, void* out, void* workspace,
                               size_t workspace_bytes, uint32_t* status_dev, void* stream);
lrkv_status lrkv_prefix_partials(const lrkv_dims* dims, const void* q, const void* BK, const lrkv_cache* cache,
                                 const int32_t* prefix_blocks, int32_t max_prefix_blocks, const int32_t* prefix_len,
                                 int32_t batch, float* partials, void* workspace, size_t workspace_bytes,
                                 uint32_t* status_dev, void* stream);

/* ======================================================================
 * Drafted tokens: a step that verifies up to 64 drafted tokens per sequence.
 *
 * The drafted tokens' rows are appended behind the sequence's own (lrkv_append, slots seq_lens[b] ..
 * seq_lens[b] + tree_lens[b] - 1), attended to by lrkv_decode_tree, and the accepted ones moved
 * together by lrkv_cache_compact; lrkv_pages_reserve and lrkv_pages_free take and give back pages.
 * ====================================================================== */
#define LRKV_MAX_TREE 64

/* Workspace bytes of lrkv_decode_tree for `batch` sequences of up to T drafted tokens, on the CURRENT device;
 * 0 for unsupported sizes. */
size_t lrkv_decode_tree_workspace_bytes(const lrkv_dims* dims, int32_t batch, int32_t T);

/*
 * lrkv_decode_tree -- Eqs. (6)-(7) for several queries per sequence: drafted token i of sequence b
 *   attends to the seq_lens[b] cached tokens and to those drafted tokens j whose bit is set in
 *   tree_mask[b][i] (usually its ancestors and itself; any set is allowed):
 *     out_{i,h} = softmax attention of q_{i,h} over these tokens, as in lrkv_decode.
 *   A query that sees no token at all gets zeros.
 *   q          [batch][T][H][d_h + d_rope]  (q^R rotated at the token's depth, e.g. by lrkv_rope)
 *   seq_lens   [batch] int32 (device), the tokens before the drafted ones; 0 is allowed
 *   tree_mask  [batch][T] uint64 (device), bit j: drafted token j is seen; bits at and behind
 *              tree_lens[b] are ignored.  NULL: a chain (token i sees j <= i)
 *   tree_lens  [batch] int32 (device) drafted tokens, 0..T; rows i >= tree_lens[b] of out are left as they
 *              were.  NULL: T for every sequence
 *   out        [batch][T][H][d_h]
 *   1 <= T <= LRKV_MAX_TREE.  A length or count outside its range (seq_lens[b] + tree_lens[b] beyond the
 *   table included) sets LRKV_DEV_BAD_SEQLEN and writes zeros to all T rows of that sequence; the tokens
 *   of a bad page id are left out (LRKV_DEV_BAD_BLOCK).  What a query does not see cannot reach its
 *   result, whatever bits it holds (NaN and infinities included), and neither can another head's latents.
 *   Probabilities enter the products with the values in bf16, q~ in two bf16 pieces; sums are fp32.
 *   Everything else as for lrkv_decode (num_splits is not used); workspace of
 *   lrkv_decode_tree_workspace_bytes(dims, batch, T) bytes, 256-byte aligned; batch x T at most 65535.
 */
lrkv_status lrkv_decode_tree(const lrkv_dims* dims, const void* q, const void* BK, const void* BV,
                             const lrkv_cache* cache, const int32_t* block_table, int32_t max_blocks_per_seq,
                             const int32_t* seq_lens, const uint64_t* tree_mask, const int32_t* tree_lens,
                             int32_t batch, int32_t T, void* out, void* workspace, size_t workspace_bytes,
                             uint32_t* status_dev, void* stream);

/* ======================================================================
 * Rotary positions of rows: queries before a decode or prefill, cached positional keys that move.
 *
 * Pair i of a head's rotated part (d_rot values) turns by position x f_i and is multiplied by
 * `magnitude`; f_i = base^(-2i / d_rot), scaled for contexts longer than the base was made for:
 *   LRKV_ROPE_NONE    as it is (with LRKV_ROPE_INTERLEAVED the rotation that lrkv_append applies)
 *   LRKV_ROPE_LINEAR  f_i / factor
 *   LRKV_ROPE_PARTS   g f_i + (1 - g) f_i / factor, g = (original_len f_i / 2 pi - low) / (high - low)
 *                     clamped to [0, 1]: pairs that turn more than `high` times over original_len
 *                     positions stay, those that turn less than `low` times are interpolated
 * ====================================================================== */
enum { LRKV_ROPE_INTERLEAVED = 0, /* pairs (2i, 2i + 1) */ LRKV_ROPE_HALF = 1 /* pairs (i, i + d_rot / 2) */ };
enum { LRKV_ROPE_NONE = 0, LRKV_ROPE_LINEAR = 1, LRKV_ROPE_PARTS = 2 };
enum { LRKV_BF16 = 0, LRKV_FP32 = 1 };

typedef struct lrkv_rope_spec {
    int32_t d_rot;       /* rotated values of a head: a multiple of 8, 8..256 */
    int32_t layout;      /* LRKV_ROPE_INTERLEAVED or LRKV_ROPE_HALF */
    int32_t scaling;     /* LRKV_ROPE_NONE, _LINEAR or _PARTS */
    int32_t reserved;    /* 0 */
    double base;         /* > 1; 0 means 10000 */
    double factor;       /* >= 1 (LINEAR, PARTS) */
    double original_len; /* > 0 (PARTS) */
    double low, high;    /* 0 <= low < high (PARTS) */
    double magnitude;    /* of the rotated values; 0 means 1 */
} lrkv_rope_spec;

/* A spec's speeds as fractions of a turn (x 2^64), filled in by lrkv_rope_make_plan; host memory, plain data. */
typedef struct lrkv_rope_plan {
    int32_t d_rot, layout;
    float magnitude;
    int32_t reserved;
    uint64_t turn[128];
} lrkv_rope_plan;

/* Host only; no device is touched. */
lrkv_status lrkv_rope_make_plan(const lrkv_rope_spec* spec, lrkv_rope_plan* plan);

/* Rows of heads: element (row, head, i) at base + row * row_stride + head * head_stride + i (strides in elements). */
typedef struct lrkv_rows {
    void* base;           /* device, 16-byte aligned */
    int64_t num_rows;     /* rows that exist; indices are checked against it */
    int64_t row_stride, head_stride; /* multiples of 8, >= 0 */
    const int32_t* index; /* [n] (device): row of the call's i-th item; negative skips it.  NULL: row i */
} lrkv_rows;

/*
 * lrkv_rope -- y_i = x_i with values [begin, begin + d_rot) of every head rotated at positions[i], i < n;
 *   the head's other values (of `width`) are copied, or not touched where x and y are the same rows.
 *   transpose = 1 applies the transposed rotation (angle -f_i x position, the same magnitude): the
 *   gradient with respect to x, and the way back where the magnitude is 1.
 *   positions   [n] int32 (device), any value (negative ones turn back: keys that move by a distance)
 *   dtype       LRKV_BF16 or LRKV_FP32, of x and y; the angle is exact modulo a turn to 2^-32 of it for any
 *               position, sine and cosine fp32, the products fp32 and rounded once
 *   width, begin  multiples of 8, begin + d_rot <= width <= 1024;  1 <= heads <= 65535
 *   x and y may be the same rows (equal struct contents: in place); otherwise no row may be read for one
 *   item and written for another.  Rows written by a call must differ from one another, and y's strides
 *   must keep its rows and heads apart.  An index at or beyond num_rows sets LRKV_DEV_BAD_SLOT and
 *   skips the item.  n == 0 is a no-op.
 */
lrkv_status lrkv_rope(const lrkv_rope_plan* plan, int32_t dtype, int32_t n, int32_t heads, int32_t width,
                      int32_t begin, const lrkv_rows* x, const lrkv_rows* y, const int32_t* positions,
                      int32_t transpose, uint32_t* status_dev, void* stream);

/* ======================================================================
 * Pages: taken, shared, copied and given back on the device, in order of the stream.
 *
 * refs [num_blocks] int32 (device, caller-owned, zeroed at first) counts for each page the table entries
 * that name it.  A page with count 0 is free.  A sequence's pages are the leading entries >= 0 of its row
 * of the block table; the entries behind them are -1.  Free pages are taken lowest first, by the
 * sequences in the order of the call, so the outcome does not depend on timing.  Counts may be raised
 * by the caller to keep pages (a shared prefix).  Calls on the same refs or tables must not overlap.
 *
 * Rows are written (lrkv_append, lrkv_cache_compact) only to pages that one sequence holds.  The pages that
 * lrkv_pages_reserve takes and the last, partly filled page of a fork are of that kind.  A sequence that is
 * cut (lrkv_pages_free with keep_lens, a smaller seq_lens) to a length inside a page that others hold too is
 * not: that page's further rows are theirs.  No call tells, as a raised count may be the caller's own.  Such
 * a sequence is forked before it goes on, and given back: the fork's last page is its own.
 * ====================================================================== */
#define LRKV_MAX_POOLS 4
#define LRKV_MAX_PAGE_BATCH 8192

/* Pools whose rows move together: the four of an lrkv_cache, the rows of an lrkv_quant_cache, the rows of a latent
 * cache, in one or several layers.  Token row t of layer l is row_bytes[p] bytes at base[p] + l layer_bytes[p] +
 * t row_bytes[p]. */
typedef struct lrkv_pools {
    void* base[LRKV_MAX_POOLS];          /* 16-byte aligned */
    int64_t row_bytes[LRKV_MAX_POOLS];   /* multiples of 16 */
    int64_t layer_bytes[LRKV_MAX_POOLS]; /* multiples of 16, >= num_blocks x 64 rows; not used with one layer */
    int32_t num_pools, num_layers, num_blocks;
} lrkv_pools;

/*
 * lrkv_pages_reserve -- pages for seq_lens[b] + new_tokens[b] tokens of every sequence: the empty entries below
 *   ceil((seq_lens[b] + new_tokens[b]) / 64) of its row are filled, those below its length included.  A
 *   sequence for whose pages too few are left gets none (LRKV_DEV_NO_PAGES) and the next one is tried; one
 *   that asks for more than its row holds, or a negative length or count, gets none (LRKV_DEV_BAD_SEQLEN),
 *   as does one with a page behind an empty entry below that bound (LRKV_DEV_BAD_BLOCK).
 *   Pages that the row already holds are taken as they are, shared ones too (see above).
 */
lrkv_status lrkv_pages_reserve(int32_t num_blocks, int32_t* refs, int32_t* block_table, int32_t max_blocks_per_seq,
                               const int32_t* seq_lens, const int32_t* new_tokens, int32_t batch,
                               uint32_t* status_dev, void* stream);

/*
 * lrkv_pages_fork -- sequence children[i] becomes a copy of sequence parents[i], i < n: what it held before is given
 *   back, its row names the parent's full pages (counts raised), and the rows of the parent's last, partly
 *   filled page are copied to a page of its own, in all pools and layers; seq_lens[child] = seq_lens[parent].
 *   Pages that the parent holds behind its length are not passed on.
 *   Where no page is left for a partly filled one, the child is left empty with length 0 (LRKV_DEV_NO_PAGES).
 *   An index out of range, a child listed twice or also listed as a parent sets LRKV_DEV_BAD_INDEX and
 *   that fork is left out; a parent's length outside its row LRKV_DEV_BAD_SEQLEN; a bad page id in the
 *   part of its row that is passed on LRKV_DEV_BAD_BLOCK (either leaves the fork out).
 */
lrkv_status lrkv_pages_fork(const lrkv_pools* pools, int32_t* refs, int32_t* block_table, int32_t max_blocks_per_seq,
                            int32_t* seq_lens, int32_t batch, const int32_t* parents, const int32_t* children,
                            int32_t n, uint32_t* status_dev, void* stream);

/*
 * lrkv_pages_free -- sequences seqs[i], i < n, give back their pages behind the first ceil(keep_lens[seqs[i]] / 64)
 *   (keep_lens [batch], or NULL: all of them): entries become -1, counts go down, and seq_lens becomes
 *   min(seq_lens, keep_lens) (0).  A sequence listed twice gives its pages back once.  A page with count 0
 *   keeps it and sets LRKV_DEV_BAD_INDEX, as does a sequence out of range; a negative keep length sets
 *   LRKV_DEV_BAD_SEQLEN and leaves that sequence alone.
 *   A keep length inside a page that other sequences hold leaves it shared: see above before rows are added.
 */
lrkv_status lrkv_pages_free(int32_t num_blocks, int32_t* refs, int32_t* block_table, int32_t max_blocks_per_seq,
                            int32_t* seq_lens, int32_t batch, const int32_t* seqs, int32_t n,
                            const int32_t* keep_lens, uint32_t* status_dev, void* stream);

/*
 * lrkv_pages_copy -- page src_pages[i] of src to page dst_pages[i] of dst, i < n, in all pools and layers (both
 *   described alike: pools, layers, row widths).  Pages written must differ from one another and from all
 *   pages read.  A negative id skips the page, one at or beyond num_blocks sets LRKV_DEV_BAD_BLOCK.
 */
lrkv_status lrkv_pages_copy(const lrkv_pools* src, const int32_t* src_pages, const lrkv_pools* dst,
                            const int32_t* dst_pages, int32_t n, uint32_t* status_dev, void* stream);

/*
 * lrkv_cache_compact -- keep the accepted ones of the tokens behind a sequence's length: row seq_lens[b] + path[b][i]
 *   moves to row seq_lens[b] + i, i < path_lens[b], in all pools and layers, and
 *   new_lens[b] = seq_lens[b] + path_lens[b]  (new_lens == NULL or == seq_lens: in place).
 *   path      [batch][max_path] int32 (device), strictly increasing and >= 0;  1 <= max_path <= 1024
 *   path_lens [batch] int32 (device), 0..max_path
 *   A path that is out of order, out of range or longer than max_path sets LRKV_DEV_BAD_INDEX, rows beyond
 *   the table or a negative length LRKV_DEV_BAD_SEQLEN, a bad page id LRKV_DEV_BAD_BLOCK; that sequence's
 *   rows stay as they are and new_lens[b] = seq_lens[b].
 *   The pages of the rows moved to must not be held by other sequences (see above).
 */
lrkv_status lrkv_cache_compact(const lrkv_pools* pools, const int32_t* block_table, int32_t max_blocks_per_seq,
                               int32_t* seq_lens, int32_t batch, const int32_t* path, const int32_t* path_lens,
                               int32_t max_path, int32_t* new_lens, uint32_t* status_dev, void* stream);

/* Workspace bytes lrkv_prefill needs (0 today; kept so callers size it). */
size_t lrkv_prefill_workspace_bytes(const lrkv_dims* dims, int32_t batch, int32_t Tq);

/*
 * lrkv_prefill -- causal chunked prefill over the cache (Eqs. (6)-(7) with the
 *   causal mask of the softmax frame): query i of sequence b sits at absolute
 *   position p = q_start[b] + i and attends to cached tokens j <= p.  The chunk's
 *   own rows must already be in the cache (lrkv_append first).
 *   Logits use the concatenated width d_h + r: [q | q~] . [s^K | z^K_h]; the
 *   scale stays 1/sqrt(d_h) (the dot product is the same one), or 1/sqrt(d_h + d_rope)
 *   with a positional key (whose term q^R . k^R joins the logit).
 *   q        [batch][Tq][H][d_h + d_rope]
 *   q_start  [batch] int32 (device)
 *   out      [batch][Tq][H][d_h]
 */
lrkv_status lrkv_prefill(const lrkv_dims* dims, const void* q, const void* BK, const void* BV,
                         const lrkv_cache* cache, const int32_t* block_table, int32_t max_blocks_per_seq,
                         const int32_t* q_start, int32_t batch, int32_t Tq, void* out, void* workspace,
                         size_t workspace_bytes, uint32_t* status_dev, void* stream);

/*
 * lrkv_prefill_fused -- lrkv_prefill with both absorptions moved into the caller's
 *   weights, as lrkv_decode_fused does for one query (associativity of frame "Compute
 *   logits without expanding historical keys", step 1, and of Eq. (7)): query i of
 *   sequence b, at absolute position p = q_start[b] + i, arrives with q~_i = q_i B_h^K
 *   already projected, and head h returns
 *     out = [ sum_{j<=p} a_j s^V_j  |  sum_{j<=p} a_j z^V_{h,j} ]   (width d_h + r),
 *     a = softmax_{j<=p}(([q_i | q~_i] . [s^K_j | z^K_{h,j}]) * scale)
 *   (with a positional key, [q | q^R | q~] . [s^K | k^R | z^K_h]).
 *   q        [batch][Tq][H][d_h + d_rope]  bf16
 *   q_tilde  [batch][Tq][H][r]             bf16, 16-byte aligned
 *   out      [batch][Tq][H][d_h + r]       bf16 (nearest, ties to even from fp32)
 *   Everything else (cache, block_table, q_start, status, errors, the stream) is as
 *   for lrkv_prefill; no B^K or B^V is read and no workspace is needed.
 */
lrkv_status lrkv_prefill_fused(const lrkv_dims* dims, const void* q, const void* q_tilde, const lrkv_cache* cache,
                               const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* q_start,
                               int32_t batch, int32_t Tq, void* out, uint32_t* status_dev, void* stream);

/* ======================================================================
 * Training-time expanded projections ("Low-Rank Key Value Attention", frame
 * "Training learns the base and residuals together": the full per-head features
 * are materialised during training).  One projection -- keys or values alike:
 *   K_h = X W_h,  W_h = W_shared + U_h B_h^T                     (Eqs. (2)-(3))
 * with its factors' gradients by the chain rule.  Dims as above (d_rope must be
 * 0; block_size and softmax_scale are not used).  Layouts:
 *   X    [n_tok][d]
 *   W_T  [d_h + H r][d]   rows: W_shared^T (d_h rows), then U_1^T .. U_H^T (r rows each)
 *   B    [H][d_h][r]
 *   Y    [n_tok][d_h + H r]  = X W_T^T = [S | R_1 .. R_H], written by the forward
 *        (bf16), read by the backward
 *   K    [n_tok][H][d_h]   = S + R_h B_h^T
 * All products on the tensor cores with fp32 accumulation; S, R and the backward's
 * [G | dR] are rounded to bf16 between the steps; outputs bf16 (nearest even).
 * n_tok == 0 is a no-op.  Every row count, d and d_h + H r are as in the ABI
 * conventions (multiples of 8); r >= 8.
 * ====================================================================== */

/* Forward: Y and K. */
lrkv_status lrkv_train_forward(const lrkv_dims* dims, const void* X, const void* W_T, const void* B, int32_t n_tok,
                               void* Y, void* K, uint32_t* status_dev, void* stream);

/* Workspace bytes lrkv_train_backward needs for n_tok rows on the CURRENT device. */
size_t lrkv_train_workspace_bytes(const lrkv_dims* dims, int32_t n_tok);

/*
 * Backward for dK [n_tok][H][d_h]:
 *   dX   [n_tok][d]       = sum_h dK_h W_h^T
 *   dW_T [d_h + H r][d]   = [dW_shared^T ; dU_1^T ; ...] = [G | dR]^T X,
 *                          G = sum_h dK_h, dR_h = dK_h B_h
 *   dB   [H][d_h][r]      = dK_h^T R_h (split over tokens, partial sums added in a
 *                          fixed order)
 *   workspace >= lrkv_train_workspace_bytes(dims, n_tok) bytes, 256-byte aligned.
 */
lrkv_status lrkv_train_backward(const lrkv_dims* dims, const void* X, const void* W_T, const void* B, const void* Y,
                                const void* dK, int32_t n_tok, void* dX, void* dW_T, void* dB, void* workspace,
                                size_t workspace_bytes, uint32_t* status_dev, void* stream);

/* ======================================================================
 * Multi-head latent attention (second workload on the same skeleton).
 *
 * "Embeddings II: MLA & Architectural Choices" (weight absorption, decoupled RoPE,
 * the softmax denominator of the concatenated width), in the associative form of
 * "Low-Rank Key Value Attention", backup frame "MLA also admits associative
 * computation": per token and layer the cache holds one row [c_t | k^R_t] -- the
 * latent c_t = x_t W^DKV (d_c = 512) and the decoupled positional key
 * k^R_t = RoPE(x_t W^KR, t) (d_rope = 64), both shared by all heads:
 *        kv : [num_blocks][block_size][d_c + d_rope]   bf16
 * With W^UK_i folded into the query and W^UV_i into the output projection, head i
 * computes  logit_t = [q~_i | q^R_i] . [c_t | k^R_t] * scale  and returns
 * o_i = sum_t softmax(logit)_t c_t (width d_c, before W^UV_i).
 * Conventions (ownership, alignment, streams, errors, status bits) as above.
 * ====================================================================== */
typedef struct lrkv_mla_dims {
    int32_t H;           /* query heads, 1..128 */
    int32_t d_c;         /* latent width; must be 512 */
    int32_t d_rope;      /* positional key width; must be 64 */
    int32_t d_head;      /* per-head content width the absorbed dot product stands for (>= 1) */
    int32_t d;           /* hidden size of appended rows; a positive multiple of 8 */
    int32_t block_size;  /* tokens per cache page; must be 64 */
    float softmax_scale; /* 0 means 1/sqrt(d_head + d_rope) */
    float rope_base;     /* RoPE base; 0 means 10000 */
} lrkv_mla_dims;

/* Bytes of one cache page: block_size * 2 * (d_c + d_rope); 0 for unsupported dims. */
size_t lrkv_mla_cache_block_bytes(const lrkv_mla_dims* dims);

/*
 * lrkv_mla_append -- write n_tok cache rows: Y = X [W^DKV | W^KR] accumulated in fp32;
 *   the last d_rope columns are rotated at positions[t] (pair (2i, 2i+1) by the angle
 *   pos * rope_base^(-2i / d_rope), computed as for lrkv_append, result rounded to
 *   fp32); then bf16 (nearest, ties to even) into slot slot_mapping[t] of kv.
 *   X            [n_tok][d]
 *   W_T          [d_c + d_rope][d]  (row c holds the weights of output column c)
 *   slot_mapping [n_tok] int32 (device); negative skips the row, >= num_blocks*block_size
 *                sets LRKV_DEV_BAD_SLOT and skips it
 *   positions    [n_tok] int32 (device), >= 0
 */
lrkv_status lrkv_mla_append(const lrkv_mla_dims* dims, const void* X, const void* W_T, int32_t n_tok,
                            const int32_t* slot_mapping, const int32_t* positions, void* kv, int32_t num_blocks,
                            uint32_t* status_dev, void* stream);

/* Workspace bytes lrkv_mla_decode needs for `batch` sequences on the CURRENT device. */
size_t lrkv_mla_decode_workspace_bytes(const lrkv_mla_dims* dims, int32_t batch);

/*
 * lrkv_mla_decode -- one decode step per sequence over all seq_lens[b] cached tokens.
 *   q           [batch][H][d_c + d_rope]  ([q~_i | q^R_i], q^R rotated by the caller)
 *   kv          [num_blocks][block_size][d_c + d_rope]
 *   block_table [batch][max_blocks_per_seq] int32 (device)
 *   seq_lens    [batch] int32 (device)
 *   out         [batch][H][d_c] bf16 (nearest, ties to even from fp32)
 *   workspace   >= lrkv_mla_decode_workspace_bytes(dims, batch) bytes, 256-byte aligned
 *   Split over the sequence across pairs of CTAs (each pair divides the row's columns),
 *   merged by log-sum-exp in a second kernel.  A sequence with a length outside
 *   [1, max_blocks_per_seq * block_size] sets LRKV_DEV_BAD_SEQLEN and gets zero rows.
 *   The call does not overlap the caller's previous kernel on the stream.
 */
lrkv_status lrkv_mla_decode(const lrkv_mla_dims* dims, const void* q, const void* kv, int32_t num_blocks,
                            const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                            int32_t batch, void* out, void* workspace, size_t workspace_bytes,
                            uint32_t* status_dev, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LRKV_H */
