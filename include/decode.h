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
 *
 * Common to all three.  16-bit tensors are float16 or bfloat16 (`dtype`, one of DECODE_F16 and
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
#define DECODE_BAD_CACHE_SLOT 2u  /* decode_qk_norm_rope: a slot outside the cache */
#define DECODE_BAD_POSITION 4u    /* decode_qk_norm_rope: a position outside the table */
#define DECODE_BAD_LENGTH 8u      /* decode_paged_attention: a length its page table cannot hold */
#define DECODE_BAD_PAGE 16u       /* decode_paged_attention: a page outside the cache */

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

/* ---- common ------------------------------------------------------------------------------------ */

/* The message of the calling thread's last failed decode_* call ("" if none). */
const char* decode_last_error(void);

/* Waits for `stream`, then reads and clears the status word of the stream's device into *bits (0: no
 * index was refused since the last read).  A device has one word for all streams and threads, and
 * a refusal is reported to whichever check comes first after it.  Returns DECODE_OK, or
 * DECODE_ERR_CUDA if the stream reported an error. */
int decode_check_status(cudaStream_t stream, uint32_t* bits);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_H */
