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
    // the states and decays that the passes hand each other.
    int64_t piece, pieces;
    float* ends;
    float* sums;
    float scale;
    int32_t nheads, ngroups, per_group, K, V;
    int32_t state_dtype, beta_f32, cu64, slot64, dst64;
    int32_t wide;      // q, k and v rows of every head 16-byte aligned
    int32_t wide_out;  // out rows of every head 8-byte aligned (fp32: 16)
    int32_t blocks;    // workgroups along V
};

constexpr float kLog2e = layer::kLog2e;

// A decay that fp32 arithmetic cannot tell from this one is taken as it: exp(-300) is 0 in
// fp32, and differences of running sums stay free of infinity minus infinity.
__device__ __forceinline__ float decay_of(float g) { return fmaxf(g, -300.f); }

// The slot named by entry `at` of a table, -1 if it is inert.
__device__ __forceinline__ int64_t slot_at(const void* table, int is64, int64_t at,
                                           const Params& p) {
    const int64_t s = load_index(table, is64, at);
    return s == p.pad_slot_id || s < 0 || s >= p.nslots ? -1 : s;
}

__device__ __forceinline__ float state_load(const void* p, int dtype, int64_t i) {
    if (dtype == SSU_F32) return static_cast<const float*>(p)[i];
    if (dtype == SSU_F16) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
    return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}

// Launchers of one io type's kernels, each in a translation unit of its own.
hipError_t step_f32(const Params& p, bool packed, hipStream_t stream);
hipError_t step_f16(const Params& p, bool packed, hipStream_t stream);
hipError_t step_bf16(const Params& p, bool packed, hipStream_t stream);
hipError_t chunk_f32(Params p, hipStream_t stream);
hipError_t chunk_f16(Params p, hipStream_t stream);
hipError_t chunk_bf16(Params p, hipStream_t stream);

}  // namespace attention
