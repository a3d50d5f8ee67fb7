/* Batched decoding over a paged local cache and a shared memory: several sequences (answers
 * sampled from one question, or several questions of one selection) attend the same selected
 * compressed memory, computed once for all of them, and each its own local K/V, which lives
 * in fixed-size pages.
 *
 * Defined by: "MSA端到端可训练记忆模型完整开源，支持亿级Token上下文", section 架构 (the selected
 * documents' compressed K/V are concatenated with the query's local K/V; 全局 RoPE: the
 * query's positions are offset by k) and section 推理流水线 step 3; MSA paper reading notes,
 * section 推理全流程 (attention context = [Top-16 compressed KV ; local KV]; the memory KV
 * stays fixed while the local KV grows).  The pages name neither batches nor paging: the
 * sequences of a group share a memory because their keys are the same for all of them.
 *
 * Packed tokens: the new tokens of all sequences lie one after another, sequence b owning
 * tokens [q_offsets[b], q_offsets[b+1]) of n_tokens.  Tokens before q_offsets[0] and from
 * q_offsets[n_seqs] on belong to nobody: nothing is stored, and q_rot and out are left as
 * they were (a batch padded to a fixed size).
 *
 * Pages: kv_pages bf16 [n_layers][n_pages][2][n_kv_heads][page_size][head_dim] (keys, then
 * values, head-contiguous rows as in msa_gather_kv's output); row r of sequence b lies in
 * page page_table[b][r / page_size], slot r % page_size, in every layer.  page_size is 16,
 * 32, 64, 128 or 256.  Entries of page_table past a sequence's last row are not read.
 *
 * seq_len[b] counts sequence b's rows WITH its new tokens, so new token i (of n_b) is row
 * seq_len[b] - n_b + i.  No call changes seq_len: a repeated call computes the same again.
 */
#ifndef MSA_PAGED_H
#define MSA_PAGED_H

#include "msa_common.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest batch of one call (the kernels keep each sequence's place in shared memory). */
#define MSA_PAGED_MAX_SEQS 1024

/* Rotates and stores the new tokens.  For token i of sequence b, with row
 * r = seq_len[b] - n_b + i and position p = rope_pos_offset + pos_offset[b] + r:
 *   page row r (keys)   = bf16(RoPE(k_new, p))    (rotate-half, angle p * theta^(-2j/d))
 *   page row r (values) = bf16(v_new)
 *   q_rot               = bf16(RoPE(q, p))
 * (the rotation in fp32 on an exactly reduced angle, one rounding to bf16).
 *   q       DEVICE [n_layers][n_tokens][n_q_heads][head_dim], NULL with q_rot NULL
 *   k_new, v_new  DEVICE [n_layers][n_tokens][n_kv_heads][head_dim]
 *           all three of in_dtype (MSA_BF16 or MSA_F32).  q_stride, k_stride, v_stride: elements
 *           from one token to the next, 0 for dense rows (heads * head_dim); a layer's tokens
 *           follow the layer before at n_tokens * stride.  So the three may be parts of one
 *           fused projection.  Strides are multiples of 16 bytes.
 *   q_offsets DEVICE int32 [n_seqs + 1]; seq_len DEVICE int32 [n_seqs]
 *   pos_offset DEVICE int32 [n_seqs] or NULL (zeros)
 *   page_table DEVICE int32 [n_seqs][max_pages]
 *   q_rot   DEVICE bf16 [n_layers][n_tokens][n_q_heads][head_dim]
 *   head_dim = 128; n_q_heads / n_kv_heads in {1, 2, 4, 8}; n_kv_heads <= 16; n_seqs <=
 *   MSA_PAGED_MAX_SEQS; q, k_new, v_new, kv_pages, q_rot 16-byte aligned; q_rot overlaps no
 *   input.
 * Device conditions: a row outside [0, max_pages * page_size) is not stored and sets
 * MSA_DEVERR_LOCAL_FULL (past the end) or MSA_DEVERR_BAD_OFFSETS (seq_len[b] < n_b); a page
 * id outside [0, n_pages) is not stored to and sets MSA_DEVERR_BAD_PAGE; q_offsets that
 * decrease or leave [0, n_tokens] set MSA_DEVERR_BAD_OFFSETS, and the tokens of such a
 * sequence are skipped.  Two tokens must not share a slot (a page written by two sequences).
 * One launch, asynchronous on `stream`, graph-capturable (lengths, tables and offsets are
 * read on the device), a programmatic dependent of the kernel before it. */
msa_status msa_paged_append(const void* q, const void* k_new, const void* v_new, msa_dtype in_dtype, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, const int32_t* q_offsets, int32_t n_tokens,
                            int32_t n_seqs, int32_t n_layers, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                            void* kv_pages, int32_t n_pages, int32_t page_size, const int32_t* page_table,
                            int32_t max_pages, const int32_t* seq_len, const int32_t* pos_offset,
                            int32_t rope_pos_offset, float rope_theta, void* q_rot, int32_t* dev_err,
                            msa_stream_t stream);

/* Workspace bytes of one msa_shared_attend call. */
msa_status msa_shared_attend_workspace_size(int32_t n_tokens, int32_t n_seqs, int32_t n_groups, int32_t n_layers,
                                            int32_t n_q_heads, int32_t n_kv_heads, size_t* bytes);

/* Attention of every new token over its group's memory and its own sequence's pages.
 * Group g holds sequences [group_offsets[g], group_offsets[g+1]); sequences outside every
 * group have no memory (n_groups = 0: plain paged attention).  For token i of sequence b of
 * group g and layer l:
 *   keys/values = mem_kv[g][l][0/1][h][0 .. mem_len[g][l]) followed by the page rows
 *                 0 .. seq_len[b] - n_b + i of sequence b (the new tokens are stored already:
 *                 msa_paged_append)
 *   out[l][t][hq] = softmax(softmax_scale * <q_hq, K_j>) . V_j, key head h = hq / G, and 0
 *                   for a token that sees no key at all
 * (fp32 scores, maxima and sums; the weights may be rounded to bf16 for the tensor cores, the
 * output is rounded to bf16).  The kernels, and with them the weights' rounding and the time, are
 * chosen from the sizes given (n_tokens, n_seqs, n_groups, heads, layers, max_mem_chunks,
 * max_pages * page_size), not from the lengths in use.
 *   q       DEVICE bf16 [n_layers][n_tokens][n_q_heads][head_dim], already rotated (q_rot)
 *   mem_kv  DEVICE bf16 [n_groups][n_layers][2][n_kv_heads][max_mem_chunks][head_dim]
 *           (msa_gather_kv output of n_groups queries); mem_len DEVICE int32 [n_groups][n_layers];
 *           both may be NULL when n_groups = 0
 *   group_offsets DEVICE int32 [n_groups + 1], NULL when n_groups = 0
 *   kv_pages, page_table, q_offsets, seq_len as above
 *   out     DEVICE bf16 [n_layers][n_tokens][n_q_heads][head_dim], not overlapping q
 *   workspace  DEVICE, >= msa_shared_attend_workspace_size bytes, 16-byte aligned, zeroed
 *           (e.g. cudaMemset) once before its first use; every call leaves it ready for the
 *           next, of any sizes.  Calls that share a workspace must not overlap on the device.
 *   head_dim = 128; n_q_heads / n_kv_heads in {1, 2, 4, 8}; n_kv_heads <= 16; n_seqs <=
 *   MSA_PAGED_MAX_SEQS; n_groups <= n_seqs; softmax_scale > 0 and finite; q, mem_kv, kv_pages,
 *   out, workspace 16-byte aligned; mem_kv and kv_pages hold fewer than 2^31 - 128 rows of
 *   head_dim each (MSA_ERR_CAPACITY where a batch takes the tensor-core kernels beyond that).
 * Device conditions: mem_len > max_mem_chunks is clamped with MSA_DEVERR_CAPACITY; seq_len
 * past max_pages * page_size is clamped with MSA_DEVERR_LOCAL_FULL; rows of a page id outside
 * [0, n_pages) are not seen (MSA_DEVERR_BAD_PAGE); q_offsets or group_offsets that decrease or
 * leave their range set MSA_DEVERR_BAD_OFFSETS and such a sequence (its output left as it
 * was) or group (no memory) is skipped, no other; where that leaves a sequence in several groups,
 * the last one's memory counts, and tokens in several sequences have undefined outputs.  Waits inside the tensor-core kernel are bounded: a timeout
 * sets MSA_DEVERR_TIMEOUT and leaves the output and the workspace undefined (zero it again).
 * Asynchronous on `stream`, graph-capturable, launched as programmatic dependents. */
msa_status msa_shared_attend(const void* q, const int32_t* q_offsets, int32_t n_tokens, int32_t n_seqs,
                             int32_t n_layers, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                             const void* mem_kv, const int32_t* mem_len, int32_t max_mem_chunks,
                             const int32_t* group_offsets, int32_t n_groups, const void* kv_pages, int32_t n_pages,
                             int32_t page_size, const int32_t* page_table, int32_t max_pages, const int32_t* seq_len,
                             float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                             int32_t* dev_err, msa_stream_t stream);

/* Kernels enqueued by the last successful call on this thread. */
int32_t msa_paged_last_launch_count(void);

const char* msa_paged_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MSA_PAGED_H */
