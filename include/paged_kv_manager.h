/*
 * paged_kv_manager.h -- the KV write path of libpaged_gqa.so: a host block
 * manager for the paged cache and the device kernels that store new tokens
 * (quantising, with the norm and rotation of a projection), read them back and
 * copy blocks.
 *
 * Sources: blocks are allocated only when a sequence needs a new one and are
 * freed when the request finishes ("The Ultimate Guide to LLM Inference
 * Optimization - Part 2", section "Paged Attention"); several sequences can
 * point at the same blocks of a shared prefix, each block carrying a
 * reference count, and when sequences diverge only the modified block is
 * copied ("Modern LLM Inference - Workloads, Bottlenecks, and Optimization
 * Techniques", section 8.2, "Prefix Sharing (Copy-on-Write)").
 *
 * Slots.  A physical slot is block * block_size + position-in-block; the K (and
 * V) row of a slot is pool[slot / block_size][slot % block_size][:, :], i.e.
 * Hkv * D contiguous elements starting at element slot * Hkv * D.
 *
 * Threading.  A manager is not thread-safe; one owner thread drives it.  The
 * device calls are asynchronous on `stream` and take device pointers.
 * Statuses are the pgd_status codes of paged_gqa.h.
 */
#ifndef PAGED_KV_MANAGER_H
#define PAGED_KV_MANAGER_H

#include <stddef.h>
#include <stdint.h>

#include "paged_gqa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pgd_kvm_s *pgd_kvm_t;

/* Extra statuses of the manager. */
enum pgd_kvm_status {
    PGD_ERR_NO_BLOCKS = 20,  /* the pool has no free block left (nothing changed) */
    PGD_ERR_NO_SEQ = 21,     /* unknown sequence id */
    PGD_ERR_SEQ_EXISTS = 22, /* sequence id already in use */
    PGD_ERR_SEQ_FULL = 23    /* sequence already holds max_blocks_per_seq blocks */
};

/*
 * A manager for a pool of `num_blocks` blocks of `block_size` tokens, serving
 * sequence ids 0 .. max_seqs-1, each holding at most max_blocks_per_seq
 * blocks.  Host memory only (no CUDA call).  All blocks start free.
 */
int pgd_kvm_create(pgd_kvm_t *out, int64_t num_blocks, int block_size, int max_seqs,
                   int max_blocks_per_seq);
int pgd_kvm_destroy(pgd_kvm_t m);

/* Start an empty sequence. */
int pgd_kvm_add_sequence(pgd_kvm_t m, int seq);

/*
 * Start `child` as a copy of `parent` that shares every block of it: no data
 * is copied, each shared block's reference count goes up by one.  The first
 * later append that writes into a shared last block copies that block first
 * (copy-on-write).
 */
int pgd_kvm_fork(pgd_kvm_t m, int parent, int child);

/* End a sequence: drop one reference from each of its blocks; blocks that
 * reach zero return to the free list. */
int pgd_kvm_free_sequence(pgd_kvm_t m, int seq);

/*
 * Reserve the next token position of each of the n sequences `seqs` (distinct
 * ids), in order.  slot_mapping[i] receives the physical slot the new token of
 * seqs[i] must be written to.  A sequence whose last block is full gets a
 * fresh block; one whose last block is shared gets a private copy of it, and
 * the pair (source block, new block) is appended to copy_src / copy_dst (room
 * for n pairs), with their count in *n_copies; those block copies must be run
 * (paged_kv_copy_blocks) before the new tokens are written.  If the pool runs
 * out of blocks, the call returns PGD_ERR_NO_BLOCKS and changes nothing.
 */
int pgd_kvm_append_slots(pgd_kvm_t m, const int *seqs, int n, int32_t *slot_mapping,
                         int32_t *copy_src, int32_t *copy_dst, int *n_copies);

/*
 * Write the block tables and lengths of sequences `seqs` for paged_gqa_decode:
 * table is [n, max_blocks] int32 (row i for seqs[i], entries past the
 * sequence's blocks set to -1), lens is [n] int32.  Requires max_blocks >= the
 * blocks any of the sequences holds.
 */
int pgd_kvm_block_tables(pgd_kvm_t m, const int *seqs, int n, int32_t *table, int max_blocks,
                         int32_t *lens);

/* Free blocks, and the reference count of one block (0 when free). */
int pgd_kvm_num_free(pgd_kvm_t m, int64_t *n_free);
int pgd_kvm_ref_count(pgd_kvm_t m, int64_t block, int *count);

/*
 * Device: copy whole blocks, K and V, from src[i] to dst[i] for i < n (device
 * int32 arrays).  Destinations must be distinct and differ from every source.
 * For 8-bit pages with a scale per block and KV head (paged_kv_pool_create_q8
 * with PGD_SCALE_PER_BLOCK) the destination blocks' K and V scale rows are
 * copied from the sources' too (the handle's scale arrays are written).
 */
int paged_kv_copy_blocks(pgd_pool_t pool, const int32_t *src, const int32_t *dst, int n,
                         void *stream);

/*
 * Device: store n new tokens.  k_new and v_new are [n, Hkv, D] in the pool's
 * dtype (8-bit pages: codes, already quantized with the scales of the blocks
 * they go to); slot_mapping is a device int32 array of n physical slots
 * (distinct, in [0, num_blocks * block_size)).  A slot out of range is skipped
 * and latches PGD_ERR_BLOCK_ID (read it with paged_gqa_get_error).
 */
int paged_kv_append(pgd_pool_t pool, const void *k_new, const void *v_new,
                    const int32_t *slot_mapping, int n, void *stream);

/*
 * Ragged batches.  The three calls below take the new tokens of B sequences as
 * packed rows: sequence b owns rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 (device
 * int32 [B + 1], ascending, cu_seqlens[B] <= total), and they are its last n_b =
 * cu_seqlens[b+1] - cu_seqlens[b] cached tokens: row i of it is the token at
 * position seq_lens[b] - n_b + i, found through block_table [B, max_blocks].  n_b may
 * be 0.  `total` is the rows the packed tensors have room for; rows past
 * cu_seqlens[B] are neither read as tokens nor written (a padded batch).  Rows are
 * [Hkv, D] (queries [Hq, D]) contiguous, `*_stride` elements apart (a view of a
 * packed projection is fine), 16-byte aligned, stride too.  Activations are float32
 * for float32 pools and bfloat16 for all others.  total = 0 or B = 0 does nothing.
 *
 * A sequence with an impossible length (cu_seqlens descending or past total, seq_lens
 * outside [0, max_blocks * block_size], more rows than cached tokens, a row's position past
 * the rotation table) latches PGD_ERR_SEQ_LEN: none of its tokens is stored and its
 * output rows are NaN.  A block id outside [0, num_blocks) latches PGD_ERR_BLOCK_ID:
 * the tokens of that block are not stored, or read back as NaN.
 */

/*
 * Device: store K and V rows in the pages, quantised as they are written.
 *   float32 and bfloat16 pages: copies.
 *   8-bit pages, scale per KV head: code = x / k_scale[h] (x times the rounded reciprocal),
 *     rounded to the nearest code (ties to even) and saturated (e4m3 +-448, int8 +-127); the
 *     scales are read only.  A scale below 2^-126 counts as 0, and scale 0 gives codes 0.
 *   8-bit pages, scale per block and KV head: the call also sets the scale of every
 *     block it writes to the largest of max|x| / 448 (127 for int8; the product with the
 *     rounded reciprocal) over the rows it stores there and, where the block already holds
 *     earlier tokens of the sequence (the first row is not at slot 0), the block's scale
 *     before the call.  If that
 *     grows the scale, the earlier tokens' codes are rounded again at the new scale (at
 *     most half a code step each time).  A block written from slot 0 on takes its scale
 *     from this call alone.  A largest magnitude whose scale would be below 2^-126 gives
 *     scale 0 and codes 0.  The handle's scale arrays are written.
 * Infinities and NaN take no part in a block's scale; an infinity saturates (where the
 * scale is 0 it counts as a NaN), a NaN is stored as the NaN code of e4m3 and
 * as 0 in int8.
 * Slots of a call must be distinct: blocks shared by several sequences are copied
 * first (paged_kv_copy_blocks), also partly filled ones that this call adds to.
 */
int paged_kv_write(pgd_pool_t pool, const void *k, int64_t k_stride, const void *v,
                   int64_t v_stride, int total, const int32_t *cu_seqlens, int B,
                   const int32_t *block_table, int max_blocks, const int32_t *seq_lens,
                   void *stream);

/*
 * Device: read the last n_b cached tokens of every sequence back as packed rows,
 * k_out and v_out [total, Hkv, D] contiguous in the activations' type; 8-bit pages
 * are dequantised (code * scale, rounded once).  A range [s, e) of a sequence is read
 * with seq_lens = e and n = e - s.
 */
int paged_kv_read(pgd_pool_t pool, void *k_out, void *v_out, int total,
                  const int32_t *cu_seqlens, int B, const int32_t *block_table, int max_blocks,
                  const int32_t *seq_lens, void *stream);

/*
 * Device: the norm of queries and keys for each head, their rotation by position, and
 * the write of K and V, in one pass.
 *   norm      y = x / sqrt(mean(x^2) + eps) * weight over the D elements of a head, for
 *             queries with q_weight and keys with k_weight ([D], weight_dtype PGD_F32 or
 *             PGD_BF16); a null weight: no norm of that side
 *   rotation  of the first rope_dim elements of every query and key head by the angles of
 *             the token's position p: rope is [rope_len, 2, rope_dim / 2] float32, cosines
 *             then sines; pairs (a, b) = elements (j, j + rope_dim / 2), or (2j, 2j + 1)
 *             with interleaved = 1, become (a cos - b sin, b cos + a sin).  rope_dim: a
 *             multiple of 16, at most D.  rope null: no rotation
 *   q, q_out  [total, Hq, D] rows; q_out may be q itself, or other columns of one packed
 *             row, but may not overlap q, k or v in any other way (PGD_ERR_ARG)
 * Everything is computed in float32 and rounded once: to q_out's type, or to the pages'
 * (8-bit codes and block scales come from the float32 values, by the rules of
 * paged_kv_write).  Values are stored as paged_kv_write stores them.
 */
int paged_qk_norm_rope_write(pgd_pool_t pool, const void *q, int64_t q_stride, void *q_out,
                             int64_t q_out_stride, int Hq, const void *k, int64_t k_stride,
                             const void *v, int64_t v_stride, int total, const void *q_weight,
                             const void *k_weight, int weight_dtype, float eps,
                             const float *rope, int rope_len, int rope_dim, int interleaved,
                             const int32_t *cu_seqlens, int B, const int32_t *block_table,
                             int max_blocks, const int32_t *seq_lens, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_KV_MANAGER_H */
