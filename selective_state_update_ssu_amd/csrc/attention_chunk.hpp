// attention_chunk.hpp -- linear attention of packed prompts by chunks, on the matrix cores.
//
// A workgroup walks one sequence's rows for one head and a slice of value columns, C
// rows at a time, with the state S (here [key, value]) in its accumulators. With G_i the
// running sum of the decays inside a chunk (inclusive), per chunk:
//     P_ij = (q_i . k_j) e^(G_i - G_j)   j <= i
//     R    = v,                           or with the delta rule the solution of
//     R_i  = beta_i (v_i - e^(G_i) S^T k_i) - sum_{j<i} A_ij R_j,
//            A_ij = beta_i e^(G_i - G_j) k_i . k_j
//     out  = scale (e^(G_i) q_i S + P R)
//     S    = e^(G_C) S + sum_j e^(G_C - G_j) k_j R_j^T
// G is summed in fp64 and kept as two floats, so that differences are exact to fp32 however
// far into the chunk. The solution goes block by block of 16 rows: the inverse of each
// diagonal block of 1 + A by forward substitution (stable where powers of A are not), the blocks
// below it as products.
//
// Precision: the matrix cores take bf16. bf16 inputs go in exactly, fp16 and fp32 ones as a high
// and a low part (fp16 exactly, fp32 to 2^-17), and so does everything derived (P, R, the
// weighted R and S): a product leaves out low x low only, and is accurate to about 2^-16 of
// its magnitudes. The triangular blocks go through the fp32 matrix instruction.
//
// Layouts (16x16 tiles, lane l, g = l / 16): an operand has the outer index at l % 16 and
// contracted indices in its registers, a result D[m][n] has n at l % 16 and m = 4 g + i in
// register i. Since a contraction may go in any order, a 32-long one is taken as {4 g + i} of one
// 16-tile and then {4 g + i} of the next: results (S, R) are then operands of the next product
// as they lie in registers. Rows of q, k and P keep each 32 entries in that order in LDS
// (one 16-byte read per operand); k and v with the rows contracted are read transposed.
#pragma once

#include "attention_common.hpp"

namespace attention {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kChunkThreads = 256;

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two floats as packed high parts and packed low parts.
__device__ __forceinline__ void split2(float a, float b, unsigned& hi, unsigned& lo) {
    const float f[2] = {a, b};
    hi = Pack<__bf16>::narrow(f);
    float h[2];
    Pack<__bf16>::widen(hi, h);
    const float r[2] = {a - h[0], b - h[1]};
    lo = Pack<__bf16>::narrow(r);
}

// The operand of two result tiles (a 32-long contraction), high and low parts.
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, u32x4& hi, u32x4& lo) {
    unsigned h[4], l[4];
    split2(a[0], a[1], h[0], l[0]);
    split2(a[2], a[3], h[1], l[1]);
    split2(b[0], b[1], h[2], l[2]);
    split2(b[2], b[3], h[3], l[3]);
    hi = u32x4{h[0], h[1], h[2], h[3]};
    lo = u32x4{l[0], l[1], l[2], l[3]};
}

// Eight consecutive values of a row, as loaded, and as high (and low) parts.
template <typename IT>
struct Seg {
    static constexpr int kWords = static_cast<int>(sizeof(IT)) * 2, kVecs = kWords / 4;
    u32x4 w[kVecs];
    __device__ __forceinline__ void load(const IT* p, bool wide, int most) {
        if (wide) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) w[i] = reinterpret_cast<const u32x4*>(p)[i];
        } else {
            typename Bits<IT>::type e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = reinterpret_cast<const typename Bits<IT>::type*>(p)[i < most ? i : most];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i > most) e[i] = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (sizeof(IT) == 4)
                    w[i / 4][i % 4] = e[i];
                else
                    w[i / 4][i % 4] = e[2 * i] | static_cast<unsigned>(e[2 * i + 1]) << 16;
            }
        }
    }
    __device__ __forceinline__ void parts(u32x4& hi, u32x4& lo) const {
        if constexpr (std::is_same<IT, __bf16>::value) {
            hi = w[0];
        } else {
            float f[8];
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                Pack<IT>::widen(w[i / 4][i % 4], &f[i * Pack<IT>::kPerWord]);
            split8(f32x4{f[0], f[1], f[2], f[3]}, f32x4{f[4], f[5], f[6], f[7]}, hi, lo);
        }
    }
};

template <typename IT, int KP, int NC, bool DELTA>
struct ChunkShape {
    static constexpr int NT = std::is_same<IT, __bf16>::value ? 1 : 2;  // parts of an input
    static constexpr int C = NT == 2 && KP == 256 ? 32 : 64;            // rows of a chunk
    static constexpr int VW = 64 * NC;                                  // columns of a slice
    static constexpr int KS = KP + 8, VS = VW + 8, PS = C + 8, AS = C + 4;  // LDS row strides
    static constexpr int CT = C / 16, KT = KP / 16, KB = KP / 32, TB = C / 32;
    struct Lds {
        unsigned short q[NT][C][KS], k[NT][C][KS], v[NT][C][VS], p[2][C][PS];
        float gh[C], gl[C], eg[C], beta[C];
        float a[DELTA ? C : 1][DELTA ? AS : 4];
    };
};

// The place of 4-block b (of 8 in 32 entries) in the order of the contraction.
__device__ __forceinline__ int place4(int b) { return b < 4 ? b * 8 : (b - 4) * 8 + 4; }

// Four rows x 16 columns per 16 lanes, transposed: lane l gets column l % 16 of its four rows.
__device__ __forceinline__ u32x2 read_transposed(const unsigned short* p) {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (lds_ptr)(const_cast<unsigned short*>(p))));
}

__device__ __forceinline__ u32x4 join(u32x2 a, u32x2 b) { return u32x4{a[0], a[1], b[0], b[1]}; }

template <typename IT, int KP, int NC, bool DELTA>
__global__ __launch_bounds__(kChunkThreads) void chunk_kernel(const Params p) {
    typedef ChunkShape<IT, KP, NC, DELTA> Shape;
    constexpr int NT = Shape::NT, C = Shape::C, CT = Shape::CT, KT = Shape::KT, KB = Shape::KB,
                  TB = Shape::TB, VW = Shape::VW;
    constexpr int QSEGS = C * KP / 8 / kChunkThreads, VSEGS = C * VW / 8 / kChunkThreads;
    __shared__ __attribute__((aligned(16))) typename Shape::Lds lds;

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);

    // Heads outermost: every XCD takes a share of the heads of every sequence, and the slices
    // and heads that read the same q and k lie side by side.
    const int64_t item = ssu::xcd_tile(blockIdx.x, gridDim.x);
    const int slice = static_cast<int>(item % p.blocks);
    const int64_t b = item / p.blocks % p.nseq;
    const int h = static_cast<int>(item / p.blocks / p.nseq);
    const int64_t begin = uniform64(load_index(p.cu, p.cu64, b));
    const int64_t end = uniform64(load_index(p.cu, p.cu64, b + 1));
    if (begin < 0 || end > p.rows || begin >= end) return;
    const int64_t slot = uniform64(p.slots ? slot_at(p.slots, p.slot64, b, p) : b);
    if (slot < 0) return;
    const int kg = h / p.per_group;
    const int v0 = slice * VW;              // first column of the slice
    const int wv = wave * 16 * NC;          // first column of the wave in it
    const int64_t n_all = end - begin;

    const IT* q = static_cast<const IT*>(p.q) + begin * p.q_stride + static_cast<int64_t>(kg) * p.K;
    const IT* k = static_cast<const IT*>(p.k) + begin * p.k_stride + static_cast<int64_t>(kg) * p.K;
    const IT* v = static_cast<const IT*>(p.v) + begin * p.v_stride + static_cast<int64_t>(h) * p.V;
    IT* out = static_cast<IT*>(p.out) + begin * p.out_stride + static_cast<int64_t>(h) * p.V;
    const float* decay = p.decay + begin * p.decay_stride + h;

    // ---- the entering state
    f32x4 S[NC][KT];
    const bool has = p.has && p.has[b];
    const int64_t in_slot = slot * p.slot_stride + static_cast<int64_t>(h) * p.V * p.K;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = v0 + wv + 16 * c + l16;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            S[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};
            const int key = 16 * t + 4 * g;
            if (has && col < p.V && key < p.K)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    S[c][t][i] = state_load(p.state, p.state_dtype,
                                            in_slot + static_cast<int64_t>(col) * p.K + key + i);
        }
    }

    // ---- what a thread moves of a chunk: its segments of q, k and v, one row's decay and beta
    Seg<IT> qr[QSEGS], kr[QSEGS], vr[VSEGS];
    float gr = 0.f, br = 0.f;
    const auto load = [&](int64_t first) {
        const int n = static_cast<int>(n_all - first < C ? n_all - first : C);
        const auto row_of = [&](int row) { return first + (row < n ? row : n - 1); };
#pragma unroll
        for (int i = 0; i < QSEGS; ++i) {
            const int s = i * kChunkThreads + tid, at = s % (KP / 8) * 8;
            const int64_t row = row_of(s / (KP / 8));
            const int c = at < p.K ? at : 0;
            qr[i].load(q + row * p.q_stride + c, p.wide & 1, 7);
            kr[i].load(k + row * p.k_stride + c, p.wide & 1, 7);
        }
#pragma unroll
        for (int i = 0; i < VSEGS; ++i) {
            const int s = i * kChunkThreads + tid, at = v0 + s % (VW / 8) * 8;
            const int c = at < p.V ? at : 0;
            vr[i].load(v + row_of(s / (VW / 8)) * p.v_stride + c, p.wide & 2,
                       p.V - 1 - c < 7 ? p.V - 1 - c : 7);
        }
        if (wave == 0) {
            const int64_t row = row_of(lane);
            gr = lane < n ? decay_of(decay[row * p.decay_stride]) : 0.f;
            if constexpr (DELTA) {
                const int64_t at = (begin + row) * p.beta_stride + h;
                const float beta = p.beta_f32 ? static_cast<const float*>(p.beta)[at]
                                              : static_cast<float>(static_cast<const IT*>(p.beta)[at]);
                br = lane < n ? beta : 0.f;
            }
        }
    };
    const auto store = [&](int64_t first) {
        const int n = static_cast<int>(n_all - first < C ? n_all - first : C);
        const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < QSEGS; ++i) {
            const int s = i * kChunkThreads + tid, seg = s % (KP / 8), row = s / (KP / 8);
            const bool in = row < n && seg * 8 < p.K;
            // Two 4-blocks of the segment's 32 entries.
            const int at = seg / 4 * 32, b0 = seg % 4 * 2;
            u32x4 part[2];
            qr[i].parts(part[0], part[1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const u32x4 x = in ? part[t] : zero;
                *reinterpret_cast<u32x2*>(&lds.q[t][row][at + place4(b0)]) = u32x2{x[0], x[1]};
                *reinterpret_cast<u32x2*>(&lds.q[t][row][at + place4(b0 + 1)]) = u32x2{x[2], x[3]};
            }
            kr[i].parts(part[0], part[1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const u32x4 x = in ? part[t] : zero;
                *reinterpret_cast<u32x2*>(&lds.k[t][row][at + place4(b0)]) = u32x2{x[0], x[1]};
                *reinterpret_cast<u32x2*>(&lds.k[t][row][at + place4(b0 + 1)]) = u32x2{x[2], x[3]};
            }
        }
#pragma unroll
        for (int i = 0; i < VSEGS; ++i) {
            const int s = i * kChunkThreads + tid, seg = s % (VW / 8), row = s / (VW / 8);
            const bool in = row < n && v0 + seg * 8 < p.V;
            u32x4 part[2];
            vr[i].parts(part[0], part[1]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                *reinterpret_cast<u32x4*>(&lds.v[t][row][seg * 8]) = in ? part[t] : zero;
        }
        if (wave == 0) {
            double G = static_cast<double>(gr) * 1.4426950408889634;
#pragma unroll
            for (int d = 1; d < C; d *= 2) {
                const double below = __shfl_up(G, d);
                if (lane >= d) G += below;
            }
            if (lane < C) {
                const float hi = static_cast<float>(G);
                lds.gh[lane] = hi;
                lds.gl[lane] = static_cast<float>(G - hi);
                lds.eg[lane] = __builtin_amdgcn_exp2f(hi);
                if constexpr (DELTA) lds.beta[lane] = br;
            }
        }
    };

    load(0);
    for (int64_t first = 0; first < n_all; first += C) {
        store(first);
        lds_barrier();
        if (first + C < n_all) load(first + C);

        // ---- scores: wave w takes row tile w
        if (wave < CT) {
            const int it = wave, i = 16 * it + l16;
            u32x4 qf[NT][KB], kf[NT][KB];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < KB; ++x) {
                    qf[t][x] = *reinterpret_cast<const u32x4*>(&lds.q[t][i][32 * x + 8 * g]);
                    if constexpr (DELTA)
                        kf[t][x] = *reinterpret_cast<const u32x4*>(&lds.k[t][i][32 * x + 8 * g]);
                }
            const float gh = lds.gh[i], gl = lds.gl[i];
            float beta = 0.f;
            if constexpr (DELTA) beta = lds.beta[i];
            for (int jt = 0; jt <= it; ++jt) {
                f32x4 s = {0.f, 0.f, 0.f, 0.f}, a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < KB; ++x) {
                    u32x4 kj[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        kj[t] = *reinterpret_cast<const u32x4*>(
                            &lds.k[t][16 * jt + l16][32 * x + 8 * g]);
                    s = mma(kj[0], qf[0][x], s);
                    if constexpr (DELTA) a = mma(kj[0], kf[0][x], a);
                    if constexpr (NT == 2) {
                        s = mma(kj[0], qf[1][x], s);
                        s = mma(kj[1], qf[0][x], s);
                        if constexpr (DELTA) {
                            a = mma(kj[0], kf[1][x], a);
                            a = mma(kj[1], kf[0][x], a);
                        }
                    }
                }
                const f32x4 jh = *reinterpret_cast<const f32x4*>(&lds.gh[16 * jt + 4 * g]);
                const f32x4 jl = *reinterpret_cast<const f32x4*>(&lds.gl[16 * jt + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * jt + 4 * g + r;
                    const float e = __builtin_amdgcn_exp2f((gh - jh[r]) + (gl - jl[r]));
                    s[r] = j <= i ? s[r] * e : 0.f;
                    if constexpr (DELTA) a[r] = j < i ? -beta * (a[r] * e) : 0.f;
                }
                u32x2 hi, lo;
                unsigned hh, ll;
                split2(s[0], s[1], hh, ll);
                hi[0] = hh, lo[0] = ll;
                split2(s[2], s[3], hh, ll);
                hi[1] = hh, lo[1] = ll;
                const int at = 32 * (jt / 2) + 8 * g + 4 * (jt % 2);
                *reinterpret_cast<u32x2*>(&lds.p[0][i][at]) = hi;
                *reinterpret_cast<u32x2*>(&lds.p[1][i][at]) = lo;
                if constexpr (DELTA) *reinterpret_cast<f32x4*>(&lds.a[i][16 * jt + 4 * g]) = a;
            }
            if (it % 2 == 0) {  // the other half of the last 32 columns lies above the diagonal
                const int at = 32 * (it / 2) + 8 * g + 4;
                *reinterpret_cast<u32x2*>(&lds.p[0][i][at]) = u32x2{0, 0};
                *reinterpret_cast<u32x2*>(&lds.p[1][i][at]) = u32x2{0, 0};
            }
            if constexpr (DELTA) {
                // The diagonal block's inverse: lane l column l % 16 of (1 + A)^-1, from -A as
                // stored. All of it is read before any of it is written.
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
                float x[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float sum = r == l16 ? 1.f : 0.f;
#pragma unroll
                    for (int m = 0; m < r; ++m)
                        sum = fmaf(lds.a[16 * it + r][16 * it + m], x[m], sum);
                    x[r] = sum;
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
                if (g == 0)
#pragma unroll
                    for (int r = 0; r < 16; ++r) lds.a[16 * it + r][16 * it + l16] = x[r];
            }
        }
        lds_barrier();

        // ---- the wave's columns
        const int n = static_cast<int>(n_all - first < C ? n_all - first : C);
        if (v0 + wv < p.V) {
            const int trow = 4 * g + l16 / 4, tcol = (l16 & 3) * 4;  // of a transposed read
            u32x4 SH[NC][KB], SL[NC][KB];
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int x = 0; x < KB; ++x)
                    split8(S[c][2 * x], S[c][2 * x + 1], SH[c][x], SL[c][x]);

            // Values as operands over the chunk's rows: parts of v, or of R.
            constexpr int RT = DELTA ? 2 : NT;
            u32x4 R[NC][TB][2];
            f32x4 W[NC][CT];  // in fp32, for the weighted ones
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    u32x2 raw[NT];
                    W[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int y = 0; y < NT; ++y) {
                        raw[y] = read_transposed(&lds.v[y][16 * t + trow][wv + 16 * c + tcol]);
                        float f[4];
                        Pack<__bf16>::widen(raw[y][0], &f[0]);
                        Pack<__bf16>::widen(raw[y][1], &f[2]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) W[c][t][r] += f[r];
                        if constexpr (!DELTA) {
                            R[c][t / 2][y][t % 2 * 2] = raw[y][0];
                            R[c][t / 2][y][t % 2 * 2 + 1] = raw[y][1];
                        }
                    }
                }
            if constexpr (DELTA) {
                // R = beta (v - e^G k S), block by block of 16 rows.
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    f32x4 acc[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int x = 0; x < KB; ++x) {
                        u32x4 kf[NT];
#pragma unroll
                        for (int y = 0; y < NT; ++y)
                            kf[y] = *reinterpret_cast<const u32x4*>(
                                &lds.k[y][16 * t + l16][32 * x + 8 * g]);
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            acc[c] = mma(kf[0], SH[c][x], acc[c]);
                            acc[c] = mma(kf[0], SL[c][x], acc[c]);
                            if constexpr (NT == 2) acc[c] = mma(kf[1], SH[c][x], acc[c]);
                        }
                    }
                    const f32x4 eg = *reinterpret_cast<const f32x4*>(&lds.eg[16 * t + 4 * g]);
                    const f32x4 be = *reinterpret_cast<const f32x4*>(&lds.beta[16 * t + 4 * g]);
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            W[c][t][r] = be[r] * (W[c][t][r] - eg[r] * acc[c][r]);
#pragma unroll
                    for (int u = 0; u <= t; ++u) {
                        const f32x4 a = *reinterpret_cast<const f32x4*>(
                            &lds.a[16 * t + l16][16 * u + 4 * g]);
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            f32x4 d = u < t ? W[c][t] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                d = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], W[c][u][r], d, 0, 0, 0);
                            W[c][t] = d;
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int x = 0; x < TB; ++x)
                        split8(W[c][2 * x], W[c][2 * x + 1], R[c][x][0], R[c][x][1]);
            }

            // out, transposed: D[value][row].
#pragma unroll
            for (int it = 0; it < CT; ++it) {
                const int i = 16 * it + l16;
                f32x4 acc[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < KB; ++x) {
                    u32x4 qf[NT];
#pragma unroll
                    for (int y = 0; y < NT; ++y)
                        qf[y] = *reinterpret_cast<const u32x4*>(&lds.q[y][i][32 * x + 8 * g]);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        acc[c] = mma(SH[c][x], qf[0], acc[c]);
                        acc[c] = mma(SL[c][x], qf[0], acc[c]);
                        if constexpr (NT == 2) acc[c] = mma(SH[c][x], qf[1], acc[c]);
                    }
                }
                const float eg = lds.eg[i];
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[c] *= eg;
#pragma unroll
                for (int x = 0; x <= it / 2; ++x) {
                    const u32x4 ph = *reinterpret_cast<const u32x4*>(&lds.p[0][i][32 * x + 8 * g]);
                    const u32x4 pl = *reinterpret_cast<const u32x4*>(&lds.p[1][i][32 * x + 8 * g]);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        acc[c] = mma(R[c][x][0], ph, acc[c]);
                        acc[c] = mma(R[c][x][0], pl, acc[c]);
                        if constexpr (RT == 2) acc[c] = mma(R[c][x][1], ph, acc[c]);
                    }
                }
                if (i < n) {
                    IT* o = out + (first + i) * p.out_stride;
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int col = v0 + wv + 16 * c + 4 * g;
                        float y[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) y[r] = p.scale * acc[c][r];
                        if (p.wide_out) {
                            if (col < p.V) Raw<IT, 4>::store(o + col, Raw<IT, 4>::narrow(y));
                        } else {
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (col + r < p.V) o[col + r] = static_cast<IT>(y[r]);
                        }
                    }
                }
            }

            // S = e^(G_C) S + k^T (weighted R).
            const float gch = lds.gh[C - 1], gcl = lds.gl[C - 1], egc = lds.eg[C - 1];
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                const f32x4 jh = *reinterpret_cast<const f32x4*>(&lds.gh[16 * t + 4 * g]);
                const f32x4 jl = *reinterpret_cast<const f32x4*>(&lds.gl[16 * t + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float w = __builtin_amdgcn_exp2f((gch - jh[r]) + (gcl - jl[r]));
#pragma unroll
                    for (int c = 0; c < NC; ++c) W[c][t][r] *= w;
                }
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int x = 0; x < TB; ++x)
                    split8(W[c][2 * x], W[c][2 * x + 1], R[c][x][0], R[c][x][1]);
#pragma unroll
                for (int t = 0; t < KT; ++t) S[c][t] *= egc;
            }
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                // 4-block (l % 4) of 16-tile t: its place in the permuted 32.
                const int at = 32 * (t / 2) + (l16 & 3) * 8 + 4 * (t % 2);
#pragma unroll
                for (int x = 0; x < TB; ++x) {
                    u32x4 kt[NT];
#pragma unroll
                    for (int y = 0; y < NT; ++y)
                        kt[y] = join(read_transposed(&lds.k[y][32 * x + trow][at]),
                                     read_transposed(&lds.k[y][32 * x + 16 + trow][at]));
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        S[c][t] = mma(kt[0], R[c][x][0], S[c][t]);
                        S[c][t] = mma(kt[0], R[c][x][1], S[c][t]);
                        if constexpr (NT == 2) S[c][t] = mma(kt[1], R[c][x][0], S[c][t]);
                    }
                }
            }
        }
        lds_barrier();
    }

    // ---- the state after the last row
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int col = v0 + wv + 16 * c + l16;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const int key = 16 * t + 4 * g;
            if (col >= p.V || key >= p.K) continue;
            const int64_t at = in_slot + static_cast<int64_t>(col) * p.K + key;
            const float s[4] = {S[c][t][0], S[c][t][1], S[c][t][2], S[c][t][3]};
            if (p.state_dtype == SSU_F32)
                Raw<float, 4>::store(static_cast<float*>(p.state) + at, Raw<float, 4>::narrow(s));
            else if (p.state_dtype == SSU_F16)
                Raw<_Float16, 4>::store(static_cast<_Float16*>(p.state) + at,
                                        Raw<_Float16, 4>::narrow(s));
            else
                Raw<__bf16, 4>::store(static_cast<__bf16*>(p.state) + at, Raw<__bf16, 4>::narrow(s));
        }
    }
}

template <typename IT, int KP, int NC>
hipError_t launch_chunk(Params p, hipStream_t stream) {
    p.blocks = (p.V + 64 * NC - 1) / (64 * NC);
    const int64_t grid = p.nseq * p.nheads * p.blocks;
    if (grid > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 blocks(static_cast<unsigned>(grid)), threads(kChunkThreads);
    if (p.beta)
        hipLaunchKernelGGL((chunk_kernel<IT, KP, NC, true>), blocks, threads, 0, stream, p);
    else
        hipLaunchKernelGGL((chunk_kernel<IT, KP, NC, false>), blocks, threads, 0, stream, p);
    return hipGetLastError();
}

template <typename IT>
hipError_t launch_chunks(const Params& p, hipStream_t stream) {
    const bool two = p.V > 64;
    if (p.K <= 64) return two ? launch_chunk<IT, 64, 2>(p, stream) : launch_chunk<IT, 64, 1>(p, stream);
    if (p.K <= 128)
        return two ? launch_chunk<IT, 128, 2>(p, stream) : launch_chunk<IT, 128, 1>(p, stream);
    return launch_chunk<IT, 256, 1>(p, stream);
}

}  // namespace attention
