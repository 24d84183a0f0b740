// attention_common.hpp -- what the kernels of linear attention (include/attention.h) share.
#pragma once

#include "attention.h"
#include "layer_common.hpp"

namespace attention {

using layer::Raw;
using ssu::Bits;
using ssu::Pack;
using ssu::Words;
using ssu::group_sum;
using ssu::lds_barrier;
using ssu::load_index;
using ssu::uniform64;
using ssu::widen_io;

struct Params {
    void* state;
    const void* q;
    const void* k;
    const void* v;
    void* out;
    const float* decay;
    const void* beta;   // NULL: no delta rule
    const void* cu;     // NULL: row b is sequence b
    const uint8_t* has; // varlen: NULL, no sequence has an initial state
    const void* slots;
    const void* na;     // packed
    const void* dst;    // packed
    int64_t nslots, slot_stride, rows, nseq, pad_slot_id;
    int64_t q_stride, k_stride, v_stride, out_stride, decay_stride, beta_stride;
    int64_t slot_seq_stride, slot_step_stride, dst_seq_stride, dst_step_stride, steps;
    // varlen: rows of a piece (0: every sequence is one piece), pieces of a call at most, and
    // what the passes hand each other: [pieces, heads, value, key] states, [pieces, heads] decays or
    // [pieces, heads, key, key] transitions.
    int64_t piece, pieces;
    float* ends;
    float* sums;
    float* moves;
    float scale;
    int32_t nheads, ngroups, per_group, K, V;
    int32_t state_dtype, beta_f32, cu64, slot64, dst64;
    int32_t wide_qk;   // q and k rows of every head 16-byte aligned
    int32_t wide;      // v and out rows too, and 64 rows of each span less than 2^31 bytes
    int32_t blocks;    // workgroups along V (and the identity's columns)
    int32_t value_blocks;
};

constexpr float kLog2e = layer::kLog2e;

// A decay that fp32 arithmetic cannot tell from this one is taken as it: exp(-300) is 0 in
// fp32, and differences of running sums stay free of infinity minus infinity.
__device__ __forceinline__ float decay_of(float g) { return fmaxf(g, -300.f); }

// A slot's id, -1 if it is inert.
__device__ __forceinline__ int64_t usable(int64_t s, const Params& p) {
    return s == p.pad_slot_id || s < 0 || s >= p.nslots ? -1 : s;
}
// The slot named by entry `at` of a table.
__device__ __forceinline__ int64_t slot_at(const void* table, int is64, int64_t at,
                                           const Params& p) {
    return usable(load_index(table, is64, at), p);
}
// The slot of sequence b where it has one.
__device__ __forceinline__ int64_t slot_of(const Params& p, int64_t b) {
    return p.slots ? slot_at(p.slots, p.slot64, b, p) : usable(b, p);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Four consecutive elements of a state at element i (a multiple of 4).
template <typename ST>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t i) {
    float f[4];
    Raw<ST, 4>::widen(Raw<ST, 4>::load(static_cast<const ST*>(p) + i), f);
    return f32x4{f[0], f[1], f[2], f[3]};
}
template <typename ST>
__device__ __forceinline__ void store4(void* p, int64_t i, f32x4 v) {
    const float f[4] = {v[0], v[1], v[2], v[3]};
    Raw<ST, 4>::store(static_cast<ST*>(p) + i, Raw<ST, 4>::narrow(f));
}
__device__ __forceinline__ f32x4 state_load4(const void* p, int dtype, int64_t i) {
    return dtype == SSU_F32 ? load4<float>(p, i)
           : dtype == SSU_F16 ? load4<_Float16>(p, i) : load4<__bf16>(p, i);
}
// Launchers of one io type's kernels, each in a translation unit of its own.
hipError_t step_f32(const Params& p, bool packed, hipStream_t stream);
hipError_t step_f16(const Params& p, bool packed, hipStream_t stream);
hipError_t step_bf16(const Params& p, bool packed, hipStream_t stream);
hipError_t chunk_f32(Params p, hipStream_t stream);
hipError_t chunk_f16(Params p, hipStream_t stream);
hipError_t chunk_bf16(Params p, hipStream_t stream);

}  // namespace attention
