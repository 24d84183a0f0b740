/*
 * attention.h -- C ABI of linear attention with a decay for each head on AMD Instinct
 * MI355X (gfx950), plain and with the delta rule, beside ssu.h, ssd.h and layer.h, with
 * their conventions (device pointers owned by the caller, `stream` a hipStream_t, an
 * ssu_status returned, ssu_last_error() names what is wrong, no allocation, no copy
 * between host and device, no synchronisation: every call may be recorded into a HIP
 * graph; the operands' GPU is the current one).
 *
 * Per row t of a sequence, head h, with key head g = h / (nheads / ngroups):
 *     S  = exp(decay[t, h]) S                       S: [value_dim, key_dim]
 *     r  = v[t, h]                                  without beta
 *     r  = beta[t, h] (v[t, h] - S k[t, g])         with beta: the delta rule
 *     S  = S + r k[t, g]^T
 *     out[t, h] = scale S q[t, g]
 * (Katharopoulos et al., "Transformers are RNNs", 2020; Sun et al., "Retentive Network",
 * 2023, for the decay; Yang et al., "Gated Delta Networks", 2024, for the delta rule.)
 * States and sums are fp32; the state is rounded once to nearest when it is stored, out
 * once when it is written. q, k, v and the decays must be finite where a sequence has
 * rows, but for decays of minus infinity, which forget the state. An infinity or NaN in a row of the
 * state makes what that row gives infinite or NaN (not always the one of the two that the formula
 * has), and nothing else.
 *
 *   ssu_attention_varlen   packed prompts, by chunks on the matrix cores; numbers enter products
 *                          as bf16 parts, accurate to about 2^-23 of the magnitudes, but for the
 *                          state that meets q on the way to a 16-bit out: to 2^-17
 *   ssu_attention_update   one row per sequence, fp32 arithmetic
 *   ssu_attention_packed   a few rows per sequence, a state stored after each (windows of
 *                          drafted tokens), slots through tables as in ssu_packed_varlen
 *
 * Slots, row ranges and preconditions are those of layer.h: an id that equals pad_slot_id
 * or lies outside [0, nslots) makes its sequence inert (nothing read or written, its out
 * rows included); an empty range of rows does nothing; a range outside [0, rows] or running
 * backwards is inert; no two sequences share a slot; out and the states overlap no other
 * operand (checked on addresses).
 */
#ifndef SSU_ATTENTION_H
#define SSU_ATTENTION_H

#include <stddef.h>

#include "ssu.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ssu_attention_args {
    uint32_t struct_size;      /* sizeof(ssu_attention_args) */
    int32_t state_dtype;       /* ssu_dtype */
    void *state;               /* [nslots, nheads, value_dim, key_dim], a slot's values dense;
                                  16-byte aligned */
    int64_t nslots;            /* >= 1 */
    int64_t slot_stride;       /* elements between slots, >= nheads * value_dim * key_dim, a
                                  multiple of 16 bytes */
    int64_t rows, nheads, ngroups; /* >= 0, >= 1, nheads % ngroups == 0 */
    int64_t key_dim, value_dim; /* 8 to 256 in steps of 8; 1 to 256 */
    const void *q, *k;         /* [rows, ngroups, key_dim], heads dense in a row */
    const void *v;             /* [rows, nheads, value_dim], heads dense in a row */
    void *out;                 /* [rows, nheads, value_dim], heads dense in a row, written */
    int64_t q_stride, k_stride, v_stride; /* elements between rows, >= 0 */
    int64_t out_stride;        /* elements between rows, >= nheads * value_dim */
    int32_t io_dtype;          /* ssu_dtype of q, k, v and out */
    int32_t beta_dtype;        /* ssu_dtype: fp32 or io_dtype */
    const float *decay;        /* natural logarithms: [rows, nheads], or [nheads] with stride 0 */
    int64_t decay_stride;      /* elements between rows, >= 0 */
    const void *beta;          /* [rows, nheads], or NULL (no delta rule) */
    int64_t beta_stride;       /* elements between rows, >= 0 */
    double scale;
    int64_t nseq;              /* >= 0; update: equal to rows */
    const void *cu_seqlens;    /* varlen, packed: [nseq + 1]; update: NULL, row b is sequence b */
    int32_t cu_dtype;          /* ssu_index_dtype of cu_seqlens and num_accepted */
    int32_t slot_dtype;        /* ssu_index_dtype of slots */
    const uint8_t *has_initial; /* varlen: [nseq] truth values, or NULL (none has); else NULL */
    /* Slots that are read (and written where dst is NULL). varlen, update: [nseq], strides
       ignored. packed: the entry b * slot_seq_stride + (num_accepted[b] - 1) * slot_step_stride.
       NULL: sequence b uses slot b. */
    const void *slots;
    int64_t slot_seq_stride, slot_step_stride; /* packed: in entries, >= 0 */
    /* packed only, else 0: as in ssu_packed_varlen. */
    const void *num_accepted;  /* [nseq] or NULL (1 each); outside [1, steps]: inert */
    const void *dst;           /* slot of the state after row t < steps of sequence b: the entry
                                  b * dst_seq_stride + t * dst_step_stride; NULL: the state after
                                  the last row goes to the slot that was read */
    int64_t dst_seq_stride, dst_step_stride; /* in entries, >= 0 */
    int32_t dst_dtype;         /* ssu_index_dtype */
    int32_t reserved;          /* 0 */
    int64_t steps;             /* table width, >= 1 when num_accepted or dst is given */
    int64_t pad_slot_id;
    void *workspace;           /* varlen: ssu_attention_workspace_bytes(...) bytes, 256-byte
                                  aligned; may be NULL if that is 0. One call at a time: its
                                  kernels hand each other states through it */
    size_t workspace_bytes;
} ssu_attention_args;

/* Scratch of a varlen call (delta: whether beta is given). Its contents need not outlive the
 * call's kernels. */
size_t ssu_attention_workspace_bytes(int64_t rows, int64_t nseq, int64_t nheads,
                                     int64_t key_dim, int64_t value_dim, int32_t delta);
int ssu_attention_varlen(const ssu_attention_args *args, void *stream);
int ssu_attention_update(const ssu_attention_args *args, void *stream);
int ssu_attention_packed(const ssu_attention_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSU_ATTENTION_H */
