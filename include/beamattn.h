/*
 * beamattn.h -- C ABI of libbeamattn.so: the operators that fill and read the
 * caches around the beam step of beamstep.h, on AMD Instinct MI355X (gfx950).
 *
 *   bs_map_blocks    block tables and slot maps from request lengths
 *   bs_kvq_write     K and V of new tokens into an 8-bit paged cache
 *   bs_kvq_read      the values that cache holds
 *   bs_kvq_reorder   bs_kv_paged_reorder for such caches
 *   bs_cache_attn    attention over such a cache: an item's shared prompt, then
 *                    every row's own positions
 *   bs_cross_attn    attention of an item's rows to its encoder's states
 *
 * A decode step of a paged search ("llm_internals" section 9.2.2, KV-cache
 * paragraph, and 9.2.4: the prompt is shared by an item's beams) runs, layer by
 * layer: bs_map_blocks once, then bs_kvq_write, bs_cache_attn and, behind an
 * encoder, bs_cross_attn; then bs_step and bs_kvq_reorder.
 *
 * Conventions are those of beamstep.h (device and host pointers, one stream
 * per handle, status codes, BS_EINVAL decided before anything is enqueued).
 * The calls without a handle are enqueued on hip_stream (NULL: the null
 * stream) of the current device. No call but the create calls allocates, none
 * synchronises but the create and destroy calls, and all can be captured into
 * a HIP graph. A handle's workspace is written and read within each call:
 * graphs that captured one handle, or calls on it, must not overlap in time.
 * dtype is a bs_dtype: BS_F32 or BS_BF16.
 */
#ifndef BEAMATTN_H
#define BEAMATTN_H

#include <stdint.h>

#include "beamstep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Block tables and slot maps from request lengths. Request b of n has
 * start = starts[b] tokens in the cache (0 when starts is NULL) and gets
 * len = lens[b] more (negative values count as 0). With bs = block_size,
 *   have = min(ceil(start / bs), max_blocks)
 *   want = min(ceil((start + len) / bs), max_blocks), at least have
 * the request takes want - have blocks from the free list, in request order:
 * entries have..want-1 of its table row become the next ids of free_blocks (-1
 * once the list is used up), entries behind them become -1, and entries below
 * have are kept. cu[b] is the sum of the lengths before b, cu[n] their total.
 * New token i of request b, at position p = start + i, gets
 *   slots[cu[b] + i] = id * bs + p % bs, id = its table row's entry p / bs,
 * and -1 where the entry is negative, past max_blocks, or the slot would not
 * fit an int32. slots[cu[n] ..] up to max_tokens are -1; tokens at or past
 * max_tokens have no slot.
 *   free_blocks  device int32 [n_free]; NULL (n_free 0): nothing is taken, the
 *                table is only read (the rows of a bs_kv_paged, say), and new
 *                positions use the entries that it holds
 *   table        device int32 [n][max_blocks]
 *   cu           device int32 [n + 1], written
 *   slots        device int32 [max_tokens], written; may be NULL when
 *                max_tokens is 0
 *   used         device int32 [1], written: the blocks asked for, the sum of
 *                want - have (more than n_free: the list ran out); 0 when
 *                free_blocks is NULL
 * Limits: n 1..65535, block_size and max_blocks >= 1, their product and
 * max_tokens at most 2^31 - 2^21; the sums of the lengths and start + len of
 * each request stay below 2^31.
 * Errors: BS_EINVAL; BS_EDEVICE. */
int bs_map_blocks(void *hip_stream, int32_t n, int32_t block_size, int32_t max_blocks,
                  const int32_t *starts, const int32_t *lens, const int32_t *free_blocks,
                  int32_t n_free, int32_t *table, int32_t *cu, int32_t *slots,
                  int32_t max_tokens, int32_t *used);

/* One layer's 8-bit paged cache: n_blocks blocks of block_size positions of
 * kv_heads heads of head_dim values, K and V alike. A value is an e4m3 number
 * (OCP FP8: 4 exponent bits, 3 fraction bits, largest 448) times its scale, a
 * power of two held in fp32 for each (block, head). Position p of block i
 * starts at i * block_stride + p * pos_stride, its heads one after the other.
 * The pools fit bs_kv_pool: a layer is two of its planes. */
typedef struct {
    void *k, *v;             /* device, e4m3 bytes                              */
    float *k_scale, *v_scale;/* device [n_blocks][kv_heads]                     */
    int32_t n_blocks;        /* >= 1, n_blocks * block_size below 2^31          */
    int32_t block_size;      /* >= 1                                            */
    int32_t kv_heads;        /* >= 1                                            */
    int32_t head_dim;        /* a multiple of 16 up to 256                      */
    int64_t block_stride;    /* bytes; both strides and the pools' addresses    */
    int64_t pos_stride;      /* are multiples of 16                             */
} bs_kvq_desc;

/* Writes the K and V rows of n_tokens new tokens into their slots (slot =
 * block * block_size + position in the block; a token whose slot is negative or
 * past the cache is skipped). The tokens of one block are neighbours in the
 * list, skipped ones apart; a list that names a block in two places leaves its
 * content undefined. A block's tokens are written in list order, run by run, a
 * run being tokens at consecutive slots. Per run, head and tensor, with amax
 * the largest finite |x| of the run,
 *   s = 2^e, e the least integer >= -100 with amax <= 448 * 2^e;
 * where the run's first token is the block's position 0, s becomes the block's
 * scale. Otherwise the larger of s and the held scale does, and if that grows
 * it, the positions below the run are rounded to the new scale. The bytes
 * behind the run stay as they are.
 * Every stored value is x / scale rounded to nearest, ties to even; a value
 * that is not finite is stored as NaN.
 *   k, v        device, dtype, rows of kv_heads * head_dim contiguous values
 *   row_stride  elements between tokens (>= kv_heads * head_dim); rows and
 *               row_stride are 16-byte aligned
 *   slots       device int32 [n_tokens], n_tokens up to 2^31 - 2^21
 * Errors: BS_EINVAL; BS_EDEVICE. */
int bs_kvq_write(void *hip_stream, const bs_kvq_desc *cache, int32_t dtype, const void *k,
                 const void *v, int64_t row_stride, const int32_t *slots, int32_t n_tokens);

/* The values at n_slots slots (any order, repeats allowed): k and v device,
 * written, [n_slots][kv_heads][head_dim] of dtype, 16-byte aligned; zeros for a
 * slot outside the cache. bf16 holds every value of the cache with a scale of
 * at least 2^-100 exactly.
 * Errors: BS_EINVAL; BS_EDEVICE. */
int bs_kvq_read(void *hip_stream, const bs_kvq_desc *cache, int32_t dtype, const int32_t *slots,
                int32_t n_slots, void *k, void *v);

/* bs_kv_paged_reorder for n_layers 8-bit caches: the block tables, the copies
 * on write of the pools' shared blocks, and the scales of every copied block.
 * Same arguments otherwise, same order of calls, on the stream of the handle.
 *   layers  host array; all of the same shape and strides, block_size that of
 *           the paged cache, n_blocks at least its batch * blocks_per_item
 *           (blocks behind those, a prompt's say, are never touched)
 * Errors: BS_EINVAL; BS_ESTATE (as bs_kv_paged_reorder); BS_ENOMEM (host);
 * BS_EDEVICE. */
int bs_kvq_reorder(bs_kv_paged *p, const bs_kvq_desc *layers, int32_t n_layers, int32_t gen_len);

/* Attention of a search's rows over an 8-bit paged cache. Query head h uses
 * kv head h / (heads / kv_heads). Row r = b*rows + w has q_len queries (1 in a
 * decode step; k in a blockwise verify, "Blockwise Parallel Decoding" section
 * 3). Query i of row r sees the prompt_lens[b] prompt positions of item b and
 * the first lens[r] - (q_len - 1) + i of the row's own positions (the last
 * q_len of them are the queries' own, each seeing those before it), and
 *   out = sum_j softmax_j(scale * q . k_j) v_j
 * in fp32 arithmetic, rounded once (the probabilities of bf16 outputs are held
 * to 2^-15). A position whose table entry is not a block of the cache (-1, out
 * of range) is not seen. A query that sees nothing, or whose scores are all
 * -inf, gives zeros, whatever the values hold. Positions past the lengths may
 * hold anything, NaN included, and so may the scales of blocks without a seen
 * position. */
typedef struct {
    int32_t batch;             /* B >= 1                                        */
    int32_t rows;              /* rows of an item (beams), >= 1;
                                  batch * rows * q_len <= 65535, and times heads
                                  at most 2^26 - 4                              */
    int32_t q_len;             /* 1..64                                         */
    int32_t heads;             /* a multiple of kv_heads, up to 65535           */
    int32_t kv_heads;          /* >= 1                                          */
    int32_t head_dim;          /* a multiple of 16 up to 256                    */
    int32_t block_size;        /* >= 1                                          */
    int32_t max_blocks;        /* entries of a row's table, >= 1; with the block
                                  size below 2^30                               */
    int32_t max_prompt_blocks; /* entries of an item's prompt table; 0: none    */
    int32_t dtype;             /* of queries and outputs                        */
    double scale;              /* from 1e-37, below 1e30                        */
} bs_cache_attn_config;

typedef struct bs_cache_attn_state bs_cache_attn_state;

/* Allocates the workspace of the split sums once, on the current device.
 * Errors: BS_EINVAL; BS_ENOMEM; BS_EDEVICE. */
int bs_cache_attn_create(const bs_cache_attn_config *cfg, void *hip_stream,
                         bs_cache_attn_state **out);

/*   q            device, dtype, [B*rows*q_len] rows of heads*head_dim values,
 *                q_stride elements apart, 16-byte aligned
 *   table        device int32 [B*rows][table_stride], table_stride >= max_blocks
 *   lens         device int32 [B*rows]: positions held, the queries' own
 *                included; taken between 0 and max_blocks * block_size
 *   prompt_table device int32 [B][max_prompt_blocks]; NULL with
 *   prompt_lens  device int32 [B], NULL: no prompt in this call
 *   out          device, dtype, [B*rows*q_len][heads][head_dim], written,
 *                16-byte aligned
 * Errors: BS_EINVAL (also a cache of another block size, head count or
 * dimension); BS_EDEVICE. */
int bs_cache_attn(bs_cache_attn_state *h, const bs_kvq_desc *cache, const void *q,
                  int64_t q_stride, const int32_t *table, int32_t table_stride,
                  const int32_t *lens, const int32_t *prompt_table, const int32_t *prompt_lens,
                  void *out);

/* Synchronises the handle's stream and frees the workspace. */
void bs_cache_attn_destroy(bs_cache_attn_state *h);

/* Attention of an item's rows (its beams, a verify's positions, or a whole
 * target) to its encoder's states, all of them seeing the same keys:
 * out = sum_j softmax_j(scale * q . k_j) v_j over j < lens[b] with
 * mask[b][j] != 0, in fp32 arithmetic, rounded once (the probabilities of bf16
 * calls are held to 2^-15, however many rows share a call). Query head h uses kv
 * head h / (heads / kv_heads). An item that sees nothing, or a query whose scores
 * are all -inf, gives zeros, whatever the values hold. Keys past the length are
 * not read; keys and values under a zero of the mask may hold anything, NaN
 * included. */
typedef struct {
    int32_t batch;     /* B >= 1                                                */
    int32_t max_rows;  /* the most query rows of an item, >= 1                  */
    int32_t heads;     /* a multiple of kv_heads                                */
    int32_t kv_heads;  /* >= 1; batch * kv_heads <= 65535                       */
    int32_t head_dim;  /* a multiple of 16 up to 256                            */
    int32_t max_keys;  /* the most keys of an item, >= 1, below 2^30            */
    int32_t dtype;     /* of queries, keys, values and outputs                  */
    double scale;      /* from 1e-37, below 1e30                                */
} bs_cross_attn_config;

typedef struct bs_cross_attn_state bs_cross_attn_state;

/* Allocates the workspace of the split sums once, on the current device.
 * Limit: batch * max_rows * heads below 2^26.
 * Errors: BS_EINVAL; BS_ENOMEM; BS_EDEVICE. */
int bs_cross_attn_create(const bs_cross_attn_config *cfg, void *hip_stream,
                         bs_cross_attn_state **out);

/* K and V of a layer: value d of head h of key j of item b is at
 * b*batch_stride + j*pos_stride + h*head_stride + d (elements). Both addresses
 * and the strides are 16-byte aligned. */
typedef struct {
    const void *k, *v;
    int64_t batch_stride, pos_stride, head_stride;
} bs_cross_kv;

/*   q         device, dtype, [B*n_rows] rows of heads*head_dim values, q_stride
 *             elements apart, 16-byte aligned
 *   n_rows    0..max_rows (0 is a no-op)
 *   n_keys    0..max_keys keys that k and v hold
 *   lens      device int32 [B], taken between 0 and n_keys; NULL: n_keys
 *   mask      device uint8 [B][mask_stride], mask_stride >= n_keys; NULL: none
 *   out       device, dtype, [B*n_rows][heads][head_dim], written, 16-byte
 *             aligned
 * Errors: BS_EINVAL; BS_EDEVICE. */
int bs_cross_attn(bs_cross_attn_state *h, const void *q, int64_t q_stride, int32_t n_rows,
                  const bs_cross_kv *kv, int32_t n_keys, const int32_t *lens,
                  const uint8_t *mask, int64_t mask_stride, void *out);

/* Synchronises the handle's stream and frees the workspace. */
void bs_cross_attn_destroy(bs_cross_attn_state *h);

#ifdef __cplusplus
}
#endif

#endif /* BEAMATTN_H */
