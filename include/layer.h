/*
 * layer.h -- C ABI of the operators around the state update in a state space
 * layer and its serving loop on AMD Instinct MI355X (gfx950), beside ssu.h and
 * ssd.h, with their conventions (device pointers owned by the caller, `stream` a
 * hipStream_t, an ssu_status returned, ssu_last_error() names what is wrong, no
 * allocation, no copy between host and device, no synchronisation: every call
 * may be recorded into a HIP graph; the operands' GPU is the current one).
 *
 *   ssu_conv1d_varlen / ssu_conv1d_update  short causal depthwise convolution
 *   ssu_scan_varlen / ssu_scan_update      selective scan with one decay per
 *                                          channel and state element
 *   ssu_cache_alloc / _adjust / _copy / _compact   slots of state caches
 *
 * Slots follow ssu.h: an id that equals pad_slot_id or lies outside [0, nslots)
 * is inert, and so is its whole sequence (nothing read or written, its out rows
 * included). Sequence b of a varlen call owns rows [cu_seqlens[b],
 * cu_seqlens[b + 1]); an empty range does nothing (its slot stays as it is), a
 * range outside [0, rows] or running backwards is inert. Device data is never
 * checked on the host. Preconditions, as in ssu.h: no two sequences share a slot,
 * cu_seqlens is non-decreasing, out and the states overlap no other operand (checked
 * on addresses; operands of one row stride may lie in disjoint columns of one buffer).
 */
#ifndef SSU_LAYER_H
#define SSU_LAYER_H

#include "ssu.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Short causal convolution. For the row at position p of a sequence, channel c,
 * with u_q the value at position q >= 0 of x, and for q < 0 the history entry
 * q + width - 1 of the sequence's slot (zero if it has no initial state):
 *     v   = bias[c] + sum_k weight[c, k] * u_{p - (width - 1) + k}
 *     out = v * sigmoid(v) when silu, else v
 * The slot then holds the sequence's last width - 1 values, oldest first. Sums
 * are fp32, products of the io dtype's values are exact in them; out is rounded
 * once to nearest, the history is copied. One launch.
 */
typedef struct ssu_conv_args {
    uint32_t struct_size;      /* sizeof(ssu_conv_args) */
    int32_t io_dtype;          /* ssu_dtype of every operand */
    void *conv_state;          /* [nslots, width - 1, dim]: channels adjacent, entries dim apart */
    int64_t nslots;            /* >= 1 */
    int64_t slot_stride;       /* elements between slots, >= (width - 1) * dim */
    const void *x;             /* [rows, dim], channels adjacent */
    int64_t x_stride;          /* elements between rows, >= 0 */
    void *out;                 /* [rows, dim], written */
    int64_t out_stride;        /* elements between rows, >= dim */
    const void *weight;        /* [dim, width] dense */
    const void *bias;          /* [dim] or NULL */
    int64_t rows, dim;         /* >= 0, >= 1 */
    int32_t width;             /* 2, 3 or 4 */
    int32_t silu;              /* nonzero: out = v * sigmoid(v) */
    const void *cu_seqlens;    /* varlen: [nseq + 1]; update: NULL, row b is sequence b */
    int32_t cu_dtype;          /* ssu_index_dtype */
    int32_t slot_dtype;        /* ssu_index_dtype of slots */
    int64_t nseq;              /* varlen: >= 0; update: equal to rows */
    const uint8_t *has_initial; /* varlen: [nseq] truth values, or NULL (none has); update: NULL */
    const void *slots;         /* [nseq] or NULL (sequence b uses slot b) */
    int64_t pad_slot_id;
} ssu_conv_args;

int ssu_conv1d_varlen(const ssu_conv_args *args, void *stream);
int ssu_conv1d_update(const ssu_conv_args *args, void *stream);

/*
 * Selective scan (Gu & Dao, "Mamba: Linear-Time Sequence Modeling with Selective
 * State Spaces", 2023, section 3). Per row t of a sequence, channel c, g = c /
 * (dim / ngroups):
 *     v    = dt[t, c] (+ dt_bias[c]);  v = log(1 + exp(v)) when dt_softplus
 *     s[n] = exp(v * A[c, n]) * s[n] + v * x[t, c] * B[t, g, n]
 *     y    = sum_n s[n] * C[t, g, n]  (+ D[c] * x[t, c])
 *     y   *= z * sigmoid(z)                            when z is given
 * from the slot's state (zero if the sequence has no initial state), which then
 * holds the state after the last row. Arithmetic and the state between rows are
 * fp32; state and out are rounded once to nearest when they are stored.
 */
typedef struct ssu_scan_args {
    uint32_t struct_size;      /* sizeof(ssu_scan_args) */
    int32_t state_dtype;       /* ssu_dtype */
    void *state;               /* [nslots, dim, dstate], a slot's values dense; 16-byte aligned */
    int64_t nslots;            /* >= 1 */
    int64_t slot_stride;       /* elements between slots, >= dim * dstate, a multiple of 16 bytes */
    int64_t rows, dim, dstate, ngroups; /* dstate 8, 16, 32, 64, 128 or 256 */
    const void *x, *z, *dt;    /* [rows, dim]; z may be NULL (no gate) */
    const void *B, *C;         /* [rows, ngroups, dstate], groups dense in a row */
    void *out;                 /* [rows, dim], written */
    int64_t x_stride, z_stride, dt_stride, B_stride, C_stride; /* elements between rows, >= 0 */
    int64_t out_stride;        /* elements between rows, >= dim */
    int32_t io_dtype;          /* ssu_dtype of x, z, B, C and out */
    int32_t dt_dtype;          /* ssu_dtype: fp32 or io_dtype */
    const float *A;            /* [dim, dstate] dense */
    const float *D;            /* [dim] or NULL */
    const float *dt_bias;      /* [dim] or NULL */
    int32_t dt_softplus;
    int32_t cu_dtype;          /* varlen: ssu_index_dtype of cu_seqlens */
    const void *cu_seqlens;    /* varlen: [nseq + 1]; update: NULL, row b is sequence b */
    int64_t nseq;              /* varlen: >= 0; update: equal to rows */
    const uint8_t *has_initial; /* varlen: [nseq] truth values, or NULL (none has); update: NULL */
    const void *slots;         /* [nseq] or NULL (sequence b uses slot b) */
    int32_t slot_dtype;        /* ssu_index_dtype */
    int32_t reserved;          /* 0 */
    int64_t pad_slot_id;
    void *workspace;           /* varlen: ssu_scan_workspace_bytes(...) bytes, 256-byte
                                  aligned; may be NULL if that is 0. One call at a time: its
                                  kernels hand each other states through it */
    size_t workspace_bytes;
} ssu_scan_args;

/* Scratch of a varlen call. Its contents need not outlive the call's kernels. */
size_t ssu_scan_workspace_bytes(int64_t rows, int64_t nseq, int64_t dim, int64_t dstate,
                                int64_t ngroups);
int ssu_scan_varlen(const ssu_scan_args *args, void *stream);
int ssu_scan_update(const ssu_scan_args *args, void *stream);

/*
 * Slots of state caches. `refcount` [nslots] int32 counts the users of each slot;
 * a slot is free at 0 and below. Every cache is a block of slots; slot ids are
 * shared by all of them (the layers of a model).
 *
 *   ssu_cache_alloc    ids[0..n) = the n lowest free slots in ascending order, one
 *                      user each; -1 where no free slot is left.
 *   ssu_cache_adjust   delta -1 (free) or +1 (retain) for each slot named in
 *                      src[0..n): a slot named twice is adjusted twice. A free slot
 *                      stays free under both; ids outside [0, nslots) are skipped.
 *   ssu_cache_copy     slot dst[i] = slot src[i] of every cache, i < n; a pair with
 *                      an id outside [0, nslots) is skipped. No slot may be both
 *                      a source and a destination of different pairs, and none a
 *                      destination twice.
 *   ssu_cache_compact  the slots in use move to the lowest ids: with k slots in
 *                      use, the ones at ids >= k go to the free ids < k, both in
 *                      ascending order, with their counts and contents.
 *                      remap[i] = the new id of slot i, -1 if it is free.
 */
typedef struct ssu_cache_block {
    void *base;                /* slot 0 */
    int64_t slot_bytes;        /* bytes of one slot, dense, >= 0 */
    int64_t stride_bytes;      /* bytes between slots, >= slot_bytes */
} ssu_cache_block;

typedef struct ssu_cache_args {
    uint32_t struct_size;      /* sizeof(ssu_cache_args) */
    int32_t delta;             /* adjust: -1 or +1 */
    int32_t *refcount;         /* [nslots]; copy: not used */
    int64_t nslots;            /* >= 0, < 2^31 */
    const ssu_cache_block *caches; /* host array; copy and compact */
    int64_t ncaches;           /* >= 0 */
    const void *src, *dst;     /* [n] slot ids; adjust: src; copy: both */
    int32_t src_dtype, dst_dtype; /* ssu_index_dtype */
    int64_t n;                 /* alloc, adjust, copy: >= 0 */
    int32_t *ids;              /* alloc: [n], written */
    int32_t *remap;            /* compact: [nslots], written */
    int32_t *plan;             /* compact: scratch of 2 * (nslots / 2) + 1 entries */
} ssu_cache_args;

int ssu_cache_alloc(const ssu_cache_args *args, void *stream);
int ssu_cache_adjust(const ssu_cache_args *args, void *stream);
int ssu_cache_copy(const ssu_cache_args *args, void *stream);
int ssu_cache_compact(const ssu_cache_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSU_LAYER_H */
