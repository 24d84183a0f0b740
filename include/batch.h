/*
 * batch.h -- C ABI of what a serving loop decides between two model steps on the GPU, beside
 * ssu.h and layer.h, with their conventions: which drafted tokens stand, and the
 * tables of a packed batch.
 *
 *   ssu_verify_drafts   accepts or rejects drafted tokens and draws the next one
 *   ssu_batch_plan      starts, row and chunk tables, slot map from the requests' lengths
 */
#ifndef SSU_BATCH_H
#define SSU_BATCH_H

#include <stddef.h>

#include "ssu.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Verification of drafted tokens (Leviathan, Kalman & Matias, "Fast Inference from
 * Transformers via Speculative Decoding", 2023, section 2.3). Sequence b owns the 1 + n rows
 * [cu_seqlens[b], cu_seqlens[b + 1]) of target, n <= window: row i < n is the target's
 * distribution p_i at the place of draft i, row n the one behind the last. q_i is the
 * distribution that draft i was drawn from; without draft_probs it is one at the draft.
 *     accepted = the number of leading drafts x_i with uniforms[b, i] q_i(x_i) < p_i(x_i)
 *     w        = max(p - q, 0) of row `accepted` if a draft was rejected there, else p;
 *                p as well where that is zero everywhere
 *     next     = the lowest token at which the running sum of w exceeds
 *                uniforms[b, window] sum(w)
 *     tokens[b] = the accepted drafts, next, then -1;  num_accepted[b] = accepted + 1
 * num_accepted is what ssu_packed_varlen and ssu_attention_packed take: the rows of the
 * sequence whose states stand. With temperature, target holds scores: p = softmax(score /
 * temperature[b]), and where temperature[b] is 0 or below, one at the largest score (the
 * lowest token of equal ones). Without it target holds probabilities, which need not sum to one.
 * Probabilities p that are not above 0 (NaN among them) and q below 0 count as 0. A q of NaN
 * rejects its draft and leaves its token out of w; a draft outside [0, vocab) is rejected; where no
 * token has any weight, next is -1. NaN scores count as minus infinity. Probabilities from scores
 * (accurate to 2^-37) and sums are fp64.
 * A range that is empty, longer than window + 1, outside [0, rows] or running backwards:
 * tokens -1, num_accepted 0; the other sequences are those of their own ranges, also where these overlap.
 */
typedef struct ssu_verify_args {
    uint32_t struct_size;      /* sizeof(ssu_verify_args) */
    int32_t target_dtype;      /* ssu_dtype */
    const void *target;        /* [rows, vocab], a row's values adjacent */
    int64_t target_stride;     /* elements between rows, >= 0 */
    int64_t rows, vocab;       /* >= 0, < 2^31; 1 to 2^31 - 2^20 - 1 */
    int64_t nseq, window;      /* >= 0; >= 0, < 2^20 */
    const void *cu_seqlens;    /* [nseq + 1] */
    int32_t cu_dtype;          /* ssu_index_dtype */
    int32_t draft_dtype;       /* ssu_index_dtype of drafts */
    const void *drafts;        /* [nseq, window] */
    int64_t draft_seq_stride, draft_step_stride; /* in entries, >= 0 */
    const void *draft_probs;   /* [nseq, window, vocab], a distribution's values adjacent, or NULL */
    int64_t probs_seq_stride, probs_step_stride; /* in elements, >= 0 */
    int32_t probs_dtype;       /* ssu_dtype */
    int32_t reserved;          /* 0 */
    const float *uniforms;     /* [nseq, window + 1] in [0, 1) */
    int64_t uniform_stride;    /* elements between sequences, >= 0 */
    const float *temperature;  /* [nseq], or NULL (target holds probabilities) */
    int32_t *tokens;           /* [nseq, window + 1] dense, written */
    int32_t *num_accepted;     /* [nseq], written */
    void *workspace;           /* ssu_verify_workspace_bytes(...) bytes, 256-byte aligned. One
                                  call at a time */
    size_t workspace_bytes;
} ssu_verify_args;

/* Scratch of a verification (scores: whether temperature is given). */
size_t ssu_verify_workspace_bytes(int64_t rows, int64_t nseq, int64_t vocab, int32_t scores);
int ssu_verify_drafts(const ssu_verify_args *args, void *stream);

/*
 * Tables of a packed batch of `nseq` requests with lengths[b] new rows each (negative: 0), one
 * request behind the other in `rows` rows:
 *   cu_seqlens[b]        first row of request b; the last entry is the total
 *   row_seq[r]           request of row r, -1 behind the last
 *   row_pos[r]           context[b] + place of the row in its request, -1 behind the last
 *   row_slots[r]         block_table[b, row_pos / block_size] * block_size + row_pos % block_size,
 *                        -1 where the table has no such column, the entry is negative or the
 *                        row has no request
 * and, with chunk_size > 0, those of ssu_ssd_prefill for requests cut into chunks of at most
 * chunk_size rows (a request without rows has one empty chunk, so that its state comes
 * back as it went in):
 *   cu_chunk_seqlens[c]  first row of chunk c; the total behind the last chunk
 *   seq_idx[c]           request of chunk c, -1 behind the last
 *   last_chunk_indices[b] the last chunk of request b, -1 if it lies past nchunks
 * At most rows / chunk_size + nseq chunks come to be while the lengths fit the rows. Outputs
 * are int32 (row_slots int64); each may be NULL. Lengths that pass `rows` in all leave the
 * requests behind it with fewer rows in the row tables than cu_seqlens says; totals must
 * stay below 2^31.
 */
typedef struct ssu_plan_args {
    uint32_t struct_size;      /* sizeof(ssu_plan_args) */
    int32_t length_dtype;      /* ssu_index_dtype of lengths */
    const void *lengths;       /* [nseq] */
    const void *context;       /* [nseq] or NULL (0 each) */
    int32_t context_dtype;     /* ssu_index_dtype */
    int32_t table_dtype;       /* ssu_index_dtype of block_table */
    int64_t nseq, rows;        /* >= 0, < 2^31 */
    int64_t chunk_size, nchunks; /* > 0 and >= 0, or 0 and 0: no chunk tables */
    const void *block_table;   /* [nseq, table_width], or NULL: no row_slots */
    int64_t table_stride;      /* entries between requests, >= 0 */
    int64_t table_width, block_size; /* >= 0, >= 1 */
    int32_t *cu_seqlens;       /* [nseq + 1] */
    int32_t *row_seq, *row_pos; /* [rows] */
    int64_t *row_slots;        /* [rows] */
    int32_t *cu_chunk_seqlens; /* [nchunks + 1] */
    int32_t *seq_idx;          /* [nchunks] */
    int32_t *last_chunk_indices; /* [nseq] */
} ssu_plan_args;

int ssu_batch_plan(const ssu_plan_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSU_BATCH_H */
