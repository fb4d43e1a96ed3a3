/*
 * decode.h -- C ABI of the operators of a decode step in libgemm_f16.so (GB300, sm_103a): what a
 * model with gated-delta-net and attention layers runs between its dense products when every
 * sequence has one (or a few) new tokens.
 *
 *   decode_gdn_step         the gated delta rule token by token on a pool of states (gdn.h has the
 *                           prefill that leaves such states)
 *   decode_qk_norm_rope     the norm of each query and key head and the position rotation in one
 *                           pass, with the write of keys and values into a paged cache
 *   decode_paged_attention  attention of one new token per sequence over the paged cache
 *   decode_quantize_cache   the write of keys and values to a paged cache of 8-bit codes with a scale
 *                           for each block of tokens and head
 *   decode_dequantize_cache the reading back of such a cache
 *   decode_paged_attention_fp8   attention of one new token per sequence over it, with a sliding
 *                           window and first tokens that stay visible
 *   decode_linear_w4        a linear layer of few tokens with 4-bit weights and group scales
 *
 * Common to all of them.  16-bit tensors are float16 or bfloat16 (`dtype`, one of DECODE_F16 and
 * DECODE_BF16, for all of a call's 16-bit tensors); sums, norms, states and softmax statistics are
 * fp32 and each 16-bit result is rounded once.  Strides are in elements; the innermost dimension
 * (head_dim) is dense, other strides of 16-bit tensors are multiples of 8 (rows are read 16 bytes at
 * a time), and pointers are 16-byte aligned; the stride of a dimension of one element is ignored.
 * Inputs may have any such stride, zero included; a written tensor's elements must not overlap, and
 * a written tensor that shares memory with another operand is refused, but where an operation says
 * that it may be an input itself.  Buffers belong to the caller and nothing is retained.
 * Calls are asynchronous on `stream` in stream order, enqueue kernel launches only (no allocation,
 * copy or synchronisation; they may be recorded into a CUDA graph once one call has run on the
 * device) and use programmatic dependent launch: every kernel waits for all earlier work on the
 * stream before it touches memory.  An empty problem (no sequence, no token) does nothing.
 *
 * Errors: DECODE_ERR_INVALID_ARG (null pointer, negative size, head counts that form no group,
 * unknown dtype or option, workspace too small, operands that share memory),
 * DECODE_ERR_UNSUPPORTED (head_dim, strides or alignment the kernels do not have, a problem too large
 * for one launch), DECODE_ERR_CUDA (a launch failed).  Nothing is enqueued on an error;
 * decode_last_error() says why.
 *
 * Indices that live in device memory (state slots, cache slots, positions, page numbers, lengths)
 * cannot be checked on the host.  The kernels check each one: an index outside its range touches no
 * memory, and sets a bit of a status word that decode_check_status() reads and clears.  What the
 * refused row gives is said at each operation.  -1 as a slot is no error: it marks an inactive row.
 */
#ifndef DECODE_H
#define DECODE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DECODE_OK 0
#define DECODE_ERR_INVALID_ARG 1
#define DECODE_ERR_UNSUPPORTED 2
#define DECODE_ERR_CUDA 3

#define DECODE_F16 0
#define DECODE_BF16 1

/* Bits of the status word. */
#define DECODE_BAD_STATE_SLOT 1u  /* decode_gdn_step: a slot of no state */
#define DECODE_BAD_CACHE_SLOT 2u  /* a slot outside the cache, or out of its block's order */
#define DECODE_BAD_POSITION 4u    /* decode_qk_norm_rope: a position outside the table */
#define DECODE_BAD_LENGTH 8u      /* an attention: a length its page table cannot hold */
#define DECODE_BAD_PAGE 16u       /* an attention: a page outside the cache */
#define DECODE_TIMED_OUT 32u      /* decode_linear_w4: a copy or product took longer than the limit, and the
                                     call's results are undefined */

/* ---- the gated delta rule, token by token ------------------------------------------------------
 *
 * For each sequence i and value head j, with S the state [dv][dk] in slot slots[i] of the pool,
 * and for its tokens t in order:
 *
 *     S' = alpha S;  u = beta (v - S' k);  S = S' + u k^T;  o = scale S q
 *
 * as gdn_prefill computes it; the last S stays in the slot.  Heads as in gdn.h: state head j reads
 * key head j / (h_v / h_k); with h_q == h_k it reads query head j / (h_v / h_k) and writes output
 * head j, with h_q a multiple of h_v query head m reads state m / (h_q / h_v) and writes output head
 * m (at most 8 query heads per state).  alpha may be any real here, 0 included.
 *
 *   q, k, v       [n][tokens][h_q / h_k / h_v][128], 16 bits, strides of the first three dimensions
 *   alpha, beta   float [n][tokens][h_v], heads dense, strides of the first two
 *   state         float [n_slots][h_v][dv][dk], dense within a slot, state_stride (a multiple of 4)
 *                 between slots; updated in place
 *   slots         int32 [n], or NULL: sequence i has slot i (then n <= n_slots).  -1 marks an
 *                 inactive sequence: no state is touched and its outputs are zero.  A slot outside
 *                 the pool is refused the same way and reported.  No two sequences of a call may
 *                 share a slot.
 *   o             [n][tokens][h_o][128], dense, 16 bits (written; h_o = max(h_q, h_v)).  It may be v
 *                 itself where that has the same shape and is dense
 */
typedef struct {
    const void* q;
    const void* k;
    const void* v;
    const float* alpha;
    const float* beta;
    float* state;
    const int32_t* slots;
    void* o;
    int64_t n, tokens, h_q, h_k, h_v, head_dim, n_slots;
    int64_t q_stride[3], k_stride[3], v_stride[3];  /* sequence, token, head */
    int64_t alpha_stride[2], beta_stride[2];        /* sequence, token */
    int64_t state_stride;
    int32_t dtype;
    float scale;
} decode_gdn_step_args;

int decode_gdn_step(const decode_gdn_step_args* args, cudaStream_t stream);

/* ---- norm and rotation of queries and keys, write to the paged cache ---------------------------
 *
 * For each token and each head x of q and k:
 *
 *     y = x / sqrt(sum_i x_i^2 / head_dim + eps) * w     DECODE_NORM_RMS (w NULL: ones)
 *     y = x / sqrt(sum_i x_i^2 + eps) * w                DECODE_NORM_L2
 *     y = x * w                                          DECODE_NORM_NONE
 *
 * then the first `rot` elements of y are rotated in pairs: pair j (0 <= j < rot / 2) is (y_j,
 * y_(rot/2 + j)), or (y_2j, y_(2j+1)) with `interleaved`, and
 *
 *     (a, b) -> (a cos - b sin, b cos + a sin),   cos = table[p][j],  sin = table[p][rot/2 + j]
 *
 * with p the token's position.  With several axes a token has one position per axis, and the pairs
 * are dealt to the axes in order: the first sections[0] pairs to axis 0, the next sections[1] to
 * axis 1 and so on.
 *
 *   q, k          [tokens][h_q / h_k][head_dim], strides of the first two dimensions
 *   v             [tokens][h_k][head_dim] (copied to v_cache; NULL when k_cache is NULL)
 *   q_weight, k_weight   [head_dim], 16 bits, dense, or NULL
 *   positions     int32 [axes][tokens], position_stride between axes (ignored with rot == 0)
 *   table         float [table_rows][rot], dense
 *   q_out         [tokens][h_q][head_dim]; k_out [tokens][h_k][head_dim].  Either may be its input
 *                 itself (same pointer and strides).  k_out is ignored when k_cache is given.
 *   k_cache, v_cache     [pages][page_size][h_k][head_dim], strides of the first three dimensions,
 *                 or both NULL
 *   slots         int32 [tokens]: the token's place, page * page_size + offset.  -1: the token's key
 *                 and value are not written.  No two tokens of a call may share a place.
 *
 * head_dim is a multiple of 8 up to 256, rot a multiple of 16 up to head_dim.  A token with a
 * position outside the table gives zeros in q_out and k_out and is not written to the cache; one
 * with a slot outside the cache is not written to it.
 */
#define DECODE_NORM_NONE 0
#define DECODE_NORM_RMS 1
#define DECODE_NORM_L2 2
#define DECODE_MAX_AXES 4

typedef struct {
    const void* q;
    const void* k;
    const void* v;
    const void* q_weight;
    const void* k_weight;
    const int32_t* positions;
    const float* table;
    void* q_out;
    void* k_out;
    void* k_cache;
    void* v_cache;
    const int32_t* slots;
    int64_t tokens, h_q, h_k, head_dim, rot, axes, table_rows, pages, page_size;
    int64_t q_stride[2], k_stride[2], v_stride[2];          /* token, head */
    int64_t q_out_stride[2], k_out_stride[2];
    int64_t k_cache_stride[3], v_cache_stride[3];           /* page, offset, head */
    int64_t position_stride;
    int32_t sections[DECODE_MAX_AXES];                      /* pairs of each axis (axes > 1) */
    int32_t dtype, norm, interleaved;
    float eps;
} decode_qk_norm_rope_args;

int decode_qk_norm_rope(const decode_qk_norm_rope_args* args, cudaStream_t stream);

/* ---- attention of one new token per sequence over the paged cache ------------------------------
 *
 * Sequence i has lens[i] tokens in the cache (its new one among them); token t lies in page
 * page_table[i][t / page_size] at offset t % page_size.  Query head m reads key and value head
 * m / (h_q / h_kv).  Over the tokens t with lens[i] - window <= t < lens[i] (all of them with
 * window == 0):
 *
 *     s_t = scale q . K_t;   lse = log sum_t exp(s_t);   o = sum_t exp(s_t - lse) V_t
 *
 * A sequence of length 0 gives o = 0 and lse = -infinity, and so does a query whose every score is
 * -infinity.
 *
 *   q             [n][h_q][head_dim], strides of the first two dimensions
 *   k_cache, v_cache     [pages][page_size][h_kv][head_dim], strides of the first three
 *   page_table    int32 [n][table_width], table_stride between rows; entries past a sequence's
 *                 length are not read
 *   lens          int32 [n]
 *   o             [n][h_q][head_dim], dense, 16 bits (written).  It may be q itself where that is dense
 *   lse           float [n][h_q], dense, or NULL (written)
 *   workspace     decode_paged_attention_workspace_bytes() bytes, 16-byte aligned; it needs no
 *                 initialisation, and calls that may overlap on the GPU need one each
 *
 * head_dim is 64, 128 or 256.  The work is split over the cache's length and joined on the device
 * from the lengths alone, so the host never reads them.  What the host does choose by, the longest
 * length possible, is table_width * page_size, or the window: a few short sequences run in one
 * launch where the table is no wider than they need (one of 500 tokens: 5.7 us), in two where it
 * is much wider (8.1 us).  Cache contents outside a sequence's tokens never reach its result,
 * whatever they hold.  An infinity or NaN in a token's value reaches that element of its heads'
 * results and no other; an infinity does so as long as the token's weight is above 2^-100 of the
 * sequence's largest, below which 0 * infinity may give NaN.  A length below 0 or above
 * table_width * page_size is refused: it counts as 0 and is reported.  A page number outside the
 * cache is refused: its tokens are not read, the sequence's result is undefined, and it is
 * reported.
 */
typedef struct {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* page_table;
    const int32_t* lens;
    void* o;
    float* lse;
    void* workspace;
    int64_t workspace_bytes;
    int64_t n, h_q, h_kv, head_dim, pages, page_size, table_width, table_stride, window;
    int64_t q_stride[2];                              /* sequence, head */
    int64_t k_stride[3], v_stride[3];                 /* page, offset, head */
    int32_t dtype;
    float scale;
} decode_paged_attention_args;

int decode_paged_attention(const decode_paged_attention_args* args, cudaStream_t stream);

/* Workspace bytes for these heads on the current device, whatever the lengths and the batch. */
int decode_paged_attention_workspace_bytes(int64_t h_q, int64_t h_kv, int64_t head_dim,
                                           size_t* bytes);

/* ---- a paged cache of 8-bit codes ---------------------------------------------------------------
 *
 * Keys and values as E4M3 codes [pages][page_size][h_k][head_dim] with one E8M0 scale for each block
 * of block_size tokens and each head, [pages][page_size / block_size][h_k]: a code c in a block of
 * scale e stands for c * 2^(e - 127), and e = 255 for NaN.  block_size divides page_size; head_dim is
 * 64, 128 or 256; strides of the codes are multiples of 16, of the scales any.
 *
 * decode_quantize_cache writes tokens' keys and values to their places.  For each block and head
 * that new tokens go to, keys and values each on their own:
 *
 *     need = the least e >= 0 with |x| <= 448 * 2^(e - 127) for all finite new elements x
 *     e'   = need, or max(need, e) where the block holds older tokens, of scale e
 *     c    = e4m3(x * 2^(127 - e')) of the new elements, rounded to nearest even
 *     c'   = e4m3(c * 2^(e - e')) of the block's other codes, where it holds older tokens and e' > e
 *
 * so a token that is larger than those before it costs them at most the codes below E4M3's
 * smallest normal number.  Where a block's new tokens begin says what it holds: the places below
 * hold older tokens, those above nothing (a block whose first place is written begins anew).  An
 * infinity or NaN becomes the code NaN, counts for no scale and touches no other element.
 *
 *   k, v          [tokens][h_k][head_dim], strides of the first two dimensions
 *   slots         int32 [tokens]: the token's place, page * page_size + offset, or -1 for none.  A
 *                 block's tokens follow one another in the call, in the order of their places without
 *                 a gap.  One that comes after a token of its block, at most 160 tokens before, and
 *                 does not continue it is refused with those that continue it and reported, as is a
 *                 slot outside the cache: neither is written.  Tokens of one block that are further
 *                 apart leave its contents undefined.
 *
 * decode_dequantize_cache gathers tokens: k and v [tokens][h_k][head_dim] receive c * 2^(e - 127), rounded
 * once to 16 bits.  Slot -1 gives zeros, and so does one outside the cache, which is reported.
 */
typedef struct {
    const void* k;
    const void* v;
    void* k_cache;
    void* v_cache;
    void* k_scale;
    void* v_scale;
    const int32_t* slots;
    int64_t tokens, h_k, head_dim, pages, page_size;
    int64_t k_stride[2], v_stride[2];                       /* token, head */
    int64_t k_cache_stride[3], v_cache_stride[3];           /* page, offset, head */
    int64_t k_scale_stride[3], v_scale_stride[3];           /* page, block, head */
    int32_t dtype, block_size;
} decode_quantize_cache_args;

int decode_quantize_cache(const decode_quantize_cache_args* args, cudaStream_t stream);

typedef struct {
    const void* k_cache;
    const void* v_cache;
    const void* k_scale;
    const void* v_scale;
    const int32_t* slots;
    void* k;
    void* v;
    int64_t tokens, h_k, head_dim, pages, page_size;
    int64_t k_stride[2], v_stride[2];                       /* token, head */
    int64_t k_cache_stride[3], v_cache_stride[3];           /* page, offset, head */
    int64_t k_scale_stride[3], v_scale_stride[3];           /* page, block, head */
    int32_t dtype, block_size;                              /* dtype: of k and v */
} decode_dequantize_cache_args;

int decode_dequantize_cache(const decode_dequantize_cache_args* args, cudaStream_t stream);

/* decode_paged_attention over such a cache: everything said there holds, with the values that the
 * codes stand for, and with a window the first `sinks` tokens stay visible: a sequence's seen tokens
 * are t < sinks and lens[i] - window <= t < lens[i] (window == 0: all, and sinks is ignored).  A
 * scale or code that stands for NaN reaches the results of its block's or token's head; those of
 * unseen tokens reach none.  Strides of pages, offsets and blocks are below 2^32.  The workspace is its
 * own: decode_paged_attention_fp8_workspace_bytes().
 *
 * What the results hold to: a token's weight is taken to 2^-22 of itself, or to 2^-32 of the largest product of
 * weight and value scale among 16 to 64 neighbours.  A weight below 2^-126 of the sequence's largest counts as
 * 0, and so does a value whose scale is below 2^-140 of its neighbours' largest.  Elements of a bfloat16 query
 * are taken to 2^-38 of its largest.  Parts of a sequence are summed in fp32 each by itself: the sum of the
 * magnitudes of any part's values must be a number of fp32, and scale * 2^(e - 127) of a seen key's block must
 * be below 2^94 (and above 2^-126, below which a score loses bits).
 */
typedef struct {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const void* k_scale;
    const void* v_scale;
    const int32_t* page_table;
    const int32_t* lens;
    void* o;
    float* lse;
    void* workspace;
    int64_t workspace_bytes;
    int64_t n, h_q, h_kv, head_dim, pages, page_size, table_width, table_stride, window, sinks;
    int64_t q_stride[2];                                    /* sequence, head */
    int64_t k_stride[3], v_stride[3];                       /* page, offset, head */
    int64_t k_scale_stride[3], v_scale_stride[3];           /* page, block, head */
    int64_t block_size;
    int32_t dtype;
    float scale;
} decode_paged_attention_fp8_args;

int decode_paged_attention_fp8(const decode_paged_attention_fp8_args* args, cudaStream_t stream);

int decode_paged_attention_fp8_workspace_bytes(int64_t h_q, int64_t h_kv, int64_t head_dim,
                                               size_t* bytes);

/* ---- a linear layer with 4-bit weights ----------------------------------------------------------
 *
 *     y[i][j] = act(bias[j] + sum_g scales[j][g] sum_{c in g} x[i][c] (code[j][c] - zeros[j][g]))
 *
 * with g over the groups of `group` neighbouring columns (the last may be shorter).  Differences of
 * codes are exact in the tensor cores' 16 bits, sums are fp32 and so are the scales' products: y is
 * rounded once.  Made for few tokens, whose time is that of reading the weights.  The sums of a group are
 * taken before its scale: with bfloat16 they must be below 2^134 in magnitude, however small the scale.
 *
 *   x             [m][k], 16 bits, x_stride (a multiple of 8) between rows
 *   codes         [n][k / 2] bytes, code_stride (a multiple of 16) between rows: byte c holds column
 *                 2 c in its lower and 2 c + 1 in its upper half
 *   scales        [n][groups], of x's type, scale_stride between rows; groups = ceil(k / group)
 *   zeros         bytes [n][groups] of 0 .. 15, zero_stride between rows, or NULL: 8 everywhere.
 *                 (of a larger byte the lower half counts)
 *   bias          [n], of x's type, dense, or NULL
 *   y             [m][n], of x's type, y_stride between rows (written)
 *
 * k and group are multiples of 32; codes, scales and zeros span less than 2^32 bytes or elements each.
 * With k == 0 the sums are 0.
 */
#define DECODE_ACT_NONE 0
#define DECODE_ACT_RELU 1
#define DECODE_ACT_GELU 2     /* x Phi(x), in its exact form */

typedef struct {
    const void* x;
    const void* codes;
    const void* scales;
    const void* zeros;
    const void* bias;
    void* y;
    int64_t m, n, k, group;
    int64_t x_stride, code_stride, scale_stride, zero_stride, y_stride;
    int32_t dtype, activation;
} decode_linear_w4_args;

int decode_linear_w4(const decode_linear_w4_args* args, cudaStream_t stream);

/* ---- common ------------------------------------------------------------------------------------ */

/* The message of the calling thread's last failed decode_* call ("" if none). */
const char* decode_last_error(void);

/* Waits for `stream`, then reads and clears the status word of the stream's device into *bits (0: no
 * index was refused since the last read).  A device has one word for all streams and threads, and
 * a refusal is reported to whichever check comes first after it.  Returns DECODE_OK, or
 * DECODE_ERR_CUDA if the stream reported an error. */
int decode_check_status(cudaStream_t stream, uint32_t* bits);

/* Limit of one wait of decode_linear_w4's kernels, for later calls of this process (ms >= 1; default 2000).
 * After one that runs out a block waits for what it has in flight, up to the limit again, writes results
 * that are none and sets DECODE_TIMED_OUT. */
int decode_set_wait_timeout_ms(uint32_t ms);

/* Testing hook, 0 = off (default).  1: decode_linear_w4's kernels never learn that the codes of a block's second
 * stage have come, or that the operands of its second chunk of 128 columns are made, so the wait for them runs
 * out.  For failure-detection tests only. */
int decode_set_fault_injection(int mode);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_H */
