// attention_step.hpp -- linear attention row by row: the decode step (one row per sequence)
// and windows of drafted tokens (a few rows, a state stored after each).
//
// A workgroup owns rows of the state [value_dim, key_dim] of one (sequence, head). Lanes
// share a row as 16-byte pieces: VEC elements per lane, LPR lanes per row (the power of two
// that holds key_dim; lanes past it idle), 64 / LPR rows per wave instruction, LOADS
// of them in flight. With a = S k, b = S q (sums over a row's lanes, of the state before its
// decay e) and c = k . q,
//     r = beta (v - e a) or v,   out = scale (e b + r c),   S = e S + r k^T,
// so that one pass over the registers serves both sums. The state crosses HBM once in
// each direction, which bounds it; a window's state stays in registers from row to row.
// 256 sequences, 32 heads of 128 x 128 in fp32, delta rule: 182 us for 1.08 GB, 5.9 TB/s; 64
// windows of up to 5 rows, a state stored after each: 107 us, 5.0 TB/s; 3 sequences: 5 us.
#pragma once

#include "attention_common.hpp"

namespace attention {

constexpr int kStepThreads = 256;

template <typename ST>
__host__ __device__ constexpr int step_vec() { return 16 / static_cast<int>(sizeof(ST)); }

// Rows of a workgroup.
__host__ __device__ constexpr int step_rows(int lpr, int loads) {
    return kStepThreads / lpr * loads;
}

// VEC elements of q or k as loaded: by 16-byte pieces (or one shorter one) where rows are
// aligned (wide), else one by one. The choice is the whole launch's.
template <typename IT, int VEC>
struct Piece {
    static constexpr int kWide = VEC * static_cast<int>(sizeof(IT)) > 16 ? 4 : VEC;
    static __device__ __forceinline__ void load(const IT* p, bool wide, float (&f)[VEC]) {
        if (wide) {
            typename Raw<IT, kWide>::type raw[VEC / kWide];
#pragma unroll
            for (int i = 0; i < VEC / kWide; ++i) raw[i] = Raw<IT, kWide>::load(p + i * kWide);
#pragma unroll
            for (int i = 0; i < VEC / kWide; ++i) {
                float h[kWide];
                Raw<IT, kWide>::widen(raw[i], h);
#pragma unroll
                for (int j = 0; j < kWide; ++j) f[i * kWide + j] = h[j];
            }
        } else {
            typename Bits<IT>::type raw[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                raw[i] = reinterpret_cast<const typename Bits<IT>::type*>(p)[i];
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = widen_io<IT>(raw[i]);
        }
    }
};

template <typename ST, typename IT, int LPR, int LOADS, bool DELTA, bool PACKED>
__global__ __launch_bounds__(kStepThreads) void step_kernel(const Params p) {
    constexpr int VEC = step_vec<ST>(), RPI = 64 / LPR, W = VEC / Pack<ST>::kPerWord;
    typedef typename Words<W>::type words_t;
    typedef typename Bits<IT>::type bits;
    const int lane = threadIdx.x & 63, sub = lane % LPR;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    // Neighbouring workgroups (blocks of a head, heads of a sequence) share an XCD.
    const int64_t tile = ssu::xcd_tile(blockIdx.x, gridDim.x);
    const int block = static_cast<int>(tile % p.blocks);
    const int64_t bh = tile / p.blocks;
    const int h = static_cast<int>(bh % p.nheads);
    const int64_t b = bh / p.nheads;

    int64_t begin = b, end = b + 1, from;
    if constexpr (PACKED) {
        begin = uniform64(load_index(p.cu, p.cu64, b));
        end = uniform64(load_index(p.cu, p.cu64, b + 1));
        if (begin < 0 || end > p.rows || begin >= end) return;
        const int64_t kept = p.na ? uniform64(load_index(p.na, p.cu64, b)) : 1;
        if (p.na && (kept < 1 || kept > p.steps)) return;
        from = p.slots ? slot_at(p.slots, p.slot64,
                                 b * p.slot_seq_stride + (kept - 1) * p.slot_step_stride, p)
                       : usable(b, p);
    } else {
        from = slot_of(p, b);
    }
    from = uniform64(from);
    if (from < 0) return;

    const int g = h / p.per_group;
    const bool in_k = sub * VEC < p.K;
    const int kk = in_k ? sub * VEC : 0;  // idle lanes read the row's start and use zeros
    int row[LOADS];
    bool active[LOADS];
    int64_t at[LOADS];  // in a slot
    const int first = block * step_rows(LPR, LOADS) + wave * (RPI * LOADS) + lane / LPR;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int v = first + i * RPI;
        active[i] = v < p.V;
        row[i] = active[i] ? v : p.V - 1;
        at[i] = (static_cast<int64_t>(h) * p.V + row[i]) * p.K + kk;
    }
    ST* state = static_cast<ST*>(p.state);
    words_t raw[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
        raw[i] = __builtin_nontemporal_load(
            reinterpret_cast<const words_t*>(state + from * p.slot_stride + at[i]));

    const IT* q = static_cast<const IT*>(p.q) + static_cast<int64_t>(g) * p.K + kk;
    const IT* k = static_cast<const IT*>(p.k) + static_cast<int64_t>(g) * p.K + kk;
    const bits* v = static_cast<const bits*>(p.v) + static_cast<int64_t>(h) * p.V;
    IT* out = static_cast<IT*>(p.out) + static_cast<int64_t>(h) * p.V;

    float S[LOADS][VEC];
    bool held = false;
    for (int64_t t = begin; t < end; ++t) {
        float qf[VEC], kf[VEC];
        bits v_in[LOADS];
        Piece<IT, VEC>::load(q + t * p.q_stride, p.wide_qk, qf);
        Piece<IT, VEC>::load(k + t * p.k_stride, p.wide_qk, kf);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) v_in[i] = v[t * p.v_stride + row[i]];
        const float e =
            __builtin_amdgcn_exp2f(kLog2e * decay_of(p.decay[t * p.decay_stride + h]));
        float beta = 1.f;
        if constexpr (DELTA) {
            const int64_t bi = t * p.beta_stride + h;
            beta = p.beta_f32 ? static_cast<const float*>(p.beta)[bi]
                              : static_cast<float>(static_cast<const IT*>(p.beta)[bi]);
        }
        int64_t to = from;
        if constexpr (PACKED) {
            if (p.dst)
                to = t - begin < p.steps
                         ? slot_at(p.dst, p.dst64,
                                   b * p.dst_seq_stride + (t - begin) * p.dst_step_stride, p)
                         : -1;
            else if (t + 1 < end)
                to = -1;
        }
        float c = 0.f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            qf[j] = in_k ? qf[j] : 0.f;
            kf[j] = in_k ? kf[j] : 0.f;
            c = fmaf(kf[j], qf[j], c);
        }
        c = group_sum<LPR>(c);
        if (!held) {
            held = true;
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
#pragma unroll
                for (int w = 0; w < W; ++w)
                    Pack<ST>::widen(raw[i][w], &S[i][w * Pack<ST>::kPerWord]);
        }
        float y[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if constexpr (DELTA) sa = fmaf(S[i][j], kf[j], sa);
                sb = fmaf(S[i][j], qf[j], sb);
            }
            if constexpr (DELTA) sa = group_sum<LPR>(sa);
            sb = group_sum<LPR>(sb);
            float r = widen_io<IT>(v_in[i]);
            if constexpr (DELTA) r = beta * (r - e * sa);
#pragma unroll
            for (int j = 0; j < VEC; ++j) S[i][j] = fmaf(r, kf[j], e * S[i][j]);
            y[i] = p.scale * fmaf(r, c, e * sb);
        }
        // Stores after all arithmetic: a load's arrival is counted together with earlier stores.
        to = uniform64(to);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            if (!active[i]) continue;
            if (to >= 0 && in_k) {
                words_t w;
#pragma unroll
                for (int j = 0; j < W; ++j) w[j] = Pack<ST>::narrow(&S[i][j * Pack<ST>::kPerWord]);
                __builtin_nontemporal_store(
                    w, reinterpret_cast<words_t*>(state + to * p.slot_stride + at[i]));
            }
            if (sub == 0) out[t * p.out_stride + row[i]] = static_cast<IT>(y[i]);
        }
    }
}

template <typename ST, typename IT, bool DELTA, bool PACKED>
hipError_t launch_step_lpr(Params p, hipStream_t stream) {
    constexpr int VEC = step_vec<ST>();
    const int pieces = (p.K + VEC - 1) / VEC;
    const auto go = [&](auto lanes) {
        constexpr int LPR = decltype(lanes)::value, LOADS = 4;
        p.blocks = (p.V + step_rows(LPR, LOADS) - 1) / step_rows(LPR, LOADS);
        const int64_t grid = p.nseq * p.nheads * p.blocks;
        if (grid > INT32_MAX) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((step_kernel<ST, IT, LPR, LOADS, DELTA, PACKED>),
                           dim3(static_cast<unsigned>(grid)), dim3(kStepThreads), 0, stream, p);
        return hipGetLastError();
    };
    if (pieces <= 2) return go(std::integral_constant<int, 2>());
    if (pieces <= 4) return go(std::integral_constant<int, 4>());
    if (pieces <= 8) return go(std::integral_constant<int, 8>());
    if (pieces <= 16) return go(std::integral_constant<int, 16>());
    if (pieces <= 32) return go(std::integral_constant<int, 32>());
    if constexpr (VEC == 4) return go(std::integral_constant<int, 64>());
    return hipErrorInvalidValue;
}

template <typename IT, bool PACKED>
hipError_t launch_step(const Params& p, hipStream_t stream) {
    const auto go = [&](auto st) {
        typedef decltype(st) ST;
        return p.beta ? launch_step_lpr<ST, IT, true, PACKED>(p, stream)
                      : launch_step_lpr<ST, IT, false, PACKED>(p, stream);
    };
    if (p.state_dtype == SSU_F32) return go(float());
    if (p.state_dtype == SSU_F16) return go(_Float16());
    return go(__bf16());
}

}  // namespace attention
