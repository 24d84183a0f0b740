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
// Where the sequences alone give too few workgroups they are cut into pieces. A first launch
// walks all but each sequence's last piece for the state alone (kEnds), a second hands
// the states on from piece to piece, and the last starts every piece from the state that enters it
// (kOut); the slot's own, which the last launch overwrites, is kept by the first. A piece changes its
// entering state to M S + N: N is what it makes of zeros. Without the delta rule M is its decay; with
// it M is what it makes of the identity as a state with no values, walked as further value columns.
//
// Precision: the matrix cores take bf16, so a number goes in as parts of 8 bits: bf16 inputs as
// one (exactly), fp16 as two (exactly), fp32 as three; what is derived (S, P, R, the weighted R) as
// three, which holds fp32's 24 bits. Products of parts whose places add up to the third's or less are
// summed: what is left out is 2^-23 of the magnitudes. Only the S that q meets goes to out in 16 bits
// as two: 2^-17 of |S| |q| is left out, where out keeps 2^-9 or 2^-12. (Three parts there as well: one
// prompt of 32,768 rows 782 us instead of 556, since its kernel has no registers left; the delta rule,
// whose S is in three anyway, 2 % more. P and R in two as well: 544 us, with the delta rule 16 prompts
// 298 instead of 309, and four times as many values of out that fp32 arithmetic rounds to the other
// side.) The triangular blocks go through the fp32 matrix instruction.
//
// Layouts (16x16 tiles, lane l, g = l / 16): an operand has the outer index at l % 16 and
// contracted indices in its registers, a result D[m][n] has n at l % 16 and m = 4 g + i in
// register i. Since a contraction may go in any order, a 32-long one is taken as {4 g + i} of one
// 16-tile and then {4 g + i} of the next: results (S, R) are then operands of the next product
// as they lie in registers. Rows of q, k and P keep each 32 entries in that order in LDS
// (one 16-byte read per operand); k and v with the rows contracted are read transposed. The
// 16-byte pieces of a row of q or k are permuted by the row (swizzle), so that neither kind of
// read meets a bank twice.
//
// Chunks of 32 rows: with 64 the triangular part doubles per row and P, A and the rows of
// two chunks (one in use, one on its way in registers) leave fewer waves; it measured no
// faster, and slower with the delta rule. What bounds it is the issue of instructions: per chunk
// and wave about 590 vector instructions for 95 matrix ones, a third of them the splitting of S,
// which every chunk needs anew. 16 prompts of 17,885 rows, 32 heads of 128 x 128 in bf16 with fp32
// states: 184-202 us (3.2-3.6 TB/s of the 655 MB that have to move; the vector units 40 % busy, matrix
// cores 25 %, LDS 20 %, and the longest prompt's workgroups outlast the rest: 1.3 waves of 2
// per SIMD on average), with the delta rule 296-318 us (40 %, 31 %, 18 %). One prompt of 32,768
// rows, 80 heads of 128 x 64: 556-574 us (a quarter of it the ends of pieces); one of 4,096 rows
// through the delta rule in fp16: 250 us (half of it the ends).
#pragma once

#include <type_traits>
#include <utility>

#include "attention_common.hpp"

namespace attention {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kChunkThreads = 256;
enum Pass { kOut, kEnds };

// Raw buffer over `bytes` bytes from `base`: loads past the range return zeros, stores past it are
// dropped. No range reaches kOutOfRange.
__device__ __forceinline__ Rsrc range_of(const void* base, unsigned bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(bytes),
                                             0x00020000);
}
constexpr unsigned kOutOfRange = 0x80000000u;

// Four consecutive elements of a state at element i of a range, as load4 and store4; i of kOutOfRange / 4
// or more lies past any.
template <typename ST>
__device__ __forceinline__ f32x4 load4(Rsrc r, unsigned i) {
    float f[4];
    if constexpr (sizeof(ST) == 4)
        Raw<ST, 4>::widen(__builtin_bit_cast(typename Raw<ST, 4>::type,
                                             __builtin_amdgcn_raw_buffer_load_b128(r, 4 * i, 0, 0)), f);
    else
        Raw<ST, 4>::widen(__builtin_bit_cast(typename Raw<ST, 4>::type,
                                             __builtin_amdgcn_raw_buffer_load_b64(r, 2 * i, 0, 0)), f);
    return f32x4{f[0], f[1], f[2], f[3]};
}
template <typename ST>
__device__ __forceinline__ void store4(Rsrc r, unsigned i, f32x4 v) {
    const float f[4] = {v[0], v[1], v[2], v[3]};
    const auto w = Raw<ST, 4>::narrow(f);
    if constexpr (sizeof(ST) == 4)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), r, 4 * i, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, w), r, 2 * i, 0, 0);
}

// f(T()) with the element type of a state.
template <typename F>
__device__ __forceinline__ void of_dtype(int dtype, F&& f) {
    if (dtype == SSU_F32)
        f(float());
    else if (dtype == SSU_F16)
        f(_Float16());
    else
        f(__bf16());
}

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two floats as the next 8-bit part of each, packed, and what the parts leave.
__device__ __forceinline__ unsigned take2(float& a, float& b) {
    const float f[2] = {a, b};
    const unsigned part = Pack<__bf16>::narrow(f);
    float h[2];
    Pack<__bf16>::widen(part, h);
    a -= h[0];
    b -= h[1];
    return part;
}

// The operands of two result tiles (a 32-long contraction), N parts.
template <int N>
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, u32x4 (&part)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
        for (int w = 0; w < 4; ++w) part[i][w] = take2(f[2 * w], f[2 * w + 1]);
        if (i + 1 < N) {
            a = f32x4{f[0], f[1], f[2], f[3]};
            b = f32x4{f[4], f[5], f[6], f[7]};
        }
    }
}

template <int N>
__device__ __forceinline__ void split4(f32x4 a, u32x2 (&part)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float f[4] = {a[0], a[1], a[2], a[3]};
        part[i] = u32x2{take2(f[0], f[1]), take2(f[2], f[3])};
        if (i + 1 < N) a = f32x4{f[0], f[1], f[2], f[3]};
    }
}

// c + a b, all products of parts whose places add up to at most LAST.
template <int LAST, int NA, int NB>
__device__ __forceinline__ f32x4 mma_parts(const u32x4 (&a)[NA], const u32x4 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (i + j <= LAST) c = mma(a[i], b[j], c);
    return c;
}

// Eight consecutive values of a row, as loaded.
template <typename IT>
struct Seg {
    static constexpr int kWords = static_cast<int>(sizeof(IT)) * 2, kVecs = kWords / 4;
    u32x4 w[kVecs];
    // At byte offset `at` of a range; zeros past its end.
    __device__ __forceinline__ void load(Rsrc r, unsigned at) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * i, 0, 0));
    }
    // The first `most` from p, one by one; zeros behind them.
    __device__ __forceinline__ void gather(const IT* p, int most) {
        typedef typename Bits<IT>::type bits;
        const bits* from = reinterpret_cast<const bits*>(p);
        bits e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < most ? from[i] : static_cast<bits>(0);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(IT) == 4)
                w[i / 4][i % 4] = e[i];
            else
                w[i / 4][i % 4] = e[2 * i] | static_cast<unsigned>(e[2 * i + 1]) << 16;
        }
    }
    template <int N>
    __device__ __forceinline__ void parts(u32x4 (&part)[N]) const {
        if constexpr (N == 1) {
            part[0] = w[0];
        } else {
            float f[8];
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                Pack<IT>::widen(w[i / 4][i % 4], &f[i * Pack<IT>::kPerWord]);
            split8(f32x4{f[0], f[1], f[2], f[3]}, f32x4{f[4], f[5], f[6], f[7]}, part);
        }
    }
};

template <typename IT, int KP, int NC, bool DELTA, Pass PASS>
struct ChunkShape {
    static constexpr bool OUT = PASS == kOut;
    static constexpr int NI = std::is_same<IT, float>::value ? 3 : std::is_same<IT, _Float16>::value ? 2 : 1;
    static constexpr int NP = 3;                                   // parts of P, with the delta rule of R
    static constexpr int NS = NI == 3 || DELTA ? 3 : 2;            // parts of S
    static constexpr int C = 32;                                   // rows of a chunk
    static constexpr int VW = 64 * NC;                             // columns of a slice
    static constexpr int CT = C / 16, KT = KP / 16, KB = KP / 32, TB = C / 32;
    // Workgroups of a compute unit (waves of a SIMD), as many as registers allow without spilling.
    static constexpr int waves(bool wide) {
        if (KP == 64) return NC == 2 ? 2 : NI == 3 || !wide ? 2 : DELTA ? 3 : 4;
        if (KP == 128) return NC == 2 || NI > 1 || DELTA ? 2 : wide ? 4 : 3;
        return NI == 1 && wide ? 2 : 1;
    }
    // LDS row strides; A keeps its 16x16 tiles on and below the diagonal.
    static constexpr int VS = VW + 8, PS = C + 8, AS = 20, TILE = 16 * AS;
    struct Lds {
        unsigned short k[NI][C][KP], v[NI][C][VS];
        unsigned short q[OUT ? NI : 1][OUT ? C : 1][OUT ? KP : 8], p[OUT ? NP : 1][OUT ? C * PS : 8];
        float gh[C], gl[C], eg[C], ew[C], beta[C];
        float a[DELTA ? CT * (CT + 1) / 2 * TILE : 4];
    };
    // Entry of P: row i, place x in the permuted order.
    static __device__ __forceinline__ int p_at(int i, int x) { return i * PS + x; }
    // Place in a row of q or k of (16-byte) piece `piece`. A 16-byte read serves lanes 0-3, 12-15 and
    // 20-27 of 32 at once, that is rows 0-3 and 12-15 of a tile with one piece and rows 4-11 with its
    // neighbour; a transposed one 4 consecutive rows with 4 neighbouring pieces: both find them at
    // 16 places.
    static __device__ __forceinline__ int piece_at(int row, int piece) {
        const int a = row >> 2 & 3, low = ((a ^ a >> 1) & 1) << 1 | a >> 1;
        return (piece ^ ((KP == 64 ? (row >> 1 & 1) << 2 : (row & 3) << 2) | low)) * 8;
    }
    static __device__ __forceinline__ int a_at(int it, int jt) { return (it * (it + 1) / 2 + jt) * TILE; }
};

// Four rows x 16 columns per 16 lanes, transposed: lane l gets column l % 16 of its four rows.
__device__ __forceinline__ u32x2 read_transposed(const unsigned short* p) {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (lds_ptr)(const_cast<unsigned short*>(p))));
}

__device__ __forceinline__ u32x4 join(u32x2 a, u32x2 b) { return u32x4{a[0], a[1], b[0], b[1]}; }

__device__ __forceinline__ u32x4 read16(const unsigned short* p) {
    return *reinterpret_cast<const u32x4*>(p);
}
// v plus what lane moves bring: one step of a running sum over the wave.
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const unsigned lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xF, false);
    const unsigned hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xF, false);
    return v + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ uint64_t lane63(uint64_t v) {
    const unsigned lo = __builtin_amdgcn_readlane(static_cast<unsigned>(v), 63);
    const unsigned hi = __builtin_amdgcn_readlane(static_cast<unsigned>(v >> 32), 63);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// Running sum over the lanes of a wave: within rows of 16 (row_shr 1, 2, 4, 8), then each row's
// last lane into the next row, then lane 31 into the upper half.
__device__ __forceinline__ double running_sum(double v) {
    v = scan_step<0x111, 0xF>(v);
    v = scan_step<0x112, 0xF>(v);
    v = scan_step<0x114, 0xF>(v);
    v = scan_step<0x118, 0xF>(v);
    v = scan_step<0x142, 0xA>(v);
    return scan_step<0x143, 0xC>(v);
}

// f(0), f(1), ... f(N - 1), each with its number as a constant.
template <int N, typename F, int... I>
__device__ __forceinline__ void unroll_each(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unroll(F&& f) {
    unroll_each<N>(f, std::make_integer_sequence<int, N>());
}

__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// The piece of a sequence that a workgroup walks.
struct Piece {
    int64_t b, begin, rows;  // sequence, first row in the call, rows
    int64_t behind;          // pieces of the sequence behind this one
    bool first, last;        // of the sequence
};

__device__ __forceinline__ int64_t rows_of(const Params& p, int64_t b, int64_t* begin) {
    const int64_t lo = load_index(p.cu, p.cu64, b), hi = load_index(p.cu, p.cu64, b + 1);
    *begin = lo;
    return lo >= 0 && hi <= p.rows && hi > lo ? hi - lo : 0;
}

// Piece `pi` of a call, by the whole wave; false if there is none. Uncut sequences of a call of
// up to 64 come longest first, so that what starts last ends soonest.
__device__ __forceinline__ bool locate(const Params& p, int64_t pi, Piece* o) {
    const int lane = threadIdx.x & 63;
    int64_t begin = 0;
    if (p.piece == 0) {
        int64_t b = pi;
        if (p.nseq > 1 && p.nseq <= 64) {
            const int64_t n = lane < p.nseq ? rows_of(p, lane, &begin) : -1;
            int rank = 0;
            for (int m = 0; m < p.nseq; ++m) {
                const int64_t other = layer::lane64(n, m);
                rank += other > n || (other == n && m < lane);
            }
            b = __builtin_ctzll(__ballot(rank == pi && lane < p.nseq));
        }
        o->b = b;
        o->rows = uniform64(rows_of(p, b, &begin));
        o->begin = uniform64(begin);
        o->behind = 0;
        o->first = o->last = true;
        return o->rows > 0;
    }
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < p.nseq; b0 += 64) {
        const int64_t b = b0 + lane;
        const int64_t n = b < p.nseq ? rows_of(p, b, &begin) : 0;
        const int mine = static_cast<int>((n + p.piece - 1) / p.piece);
        int run = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int below = __shfl_up(run, d);
            if (lane >= d) run += below;
        }
        const uint64_t behind = __ballot(before + run > pi);
        if (behind) {
            const int at = __builtin_ctzll(behind);
            const int64_t rows = layer::lane64(n, at);
            const int64_t j = pi - before - (__builtin_amdgcn_readlane(run, at) -
                                             __builtin_amdgcn_readlane(mine, at));
            o->b = b0 + at;
            o->begin = layer::lane64(begin, at) + j * p.piece;
            o->behind = __builtin_amdgcn_readlane(mine, at) - 1 - j;
            o->first = j == 0;
            o->last = (j + 1) * p.piece >= rows;
            o->rows = o->last ? rows - j * p.piece : p.piece;
            return true;
        }
        before += __builtin_amdgcn_readlane(run, 63);
    }
    return false;
}

// WIDE: rows of q, k, v and out are 16-byte aligned and a chunk's rows span less than 2^31
// bytes, so that whole pieces move through ranges that end with the chunk's rows.
template <typename IT, int KP, int NC, bool DELTA, bool WIDE, Pass PASS>
__global__ __launch_bounds__(kChunkThreads, (ChunkShape<IT, KP, NC, DELTA, PASS>::waves(WIDE)))
void chunk_kernel(const Params p) {
    typedef ChunkShape<IT, KP, NC, DELTA, PASS> Shape;
    constexpr bool OUT = PASS == kOut;
    constexpr int NI = Shape::NI, NP = Shape::NP, NS = Shape::NS, C = Shape::C, CT = Shape::CT,
                  KT = Shape::KT, KB = Shape::KB, TB = Shape::TB, VW = Shape::VW;
    constexpr int QSEGS = C * KP / 8 / kChunkThreads, VSEGS = C * VW / 8 / kChunkThreads;
    constexpr int QROWS = kChunkThreads / (KP / 8), VROWS = kChunkThreads / (VW / 8);
    constexpr unsigned ES = sizeof(IT);
    __shared__ __attribute__((aligned(16))) typename Shape::Lds lds;

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);

    // Every XCD takes a share of the heads of every piece, one piece after the other: what runs at a
    // time reads neighbouring columns of the same rows, and the slices and heads of one q and k
    // lie side by side.
    const int per_piece = p.nheads * p.blocks;
    const int64_t item = ssu::xcd_split(blockIdx.x, gridDim.x, per_piece);
    const int64_t pi = item / per_piece;
    const int h = static_cast<int>(item % per_piece) / p.blocks, slice = static_cast<int>(item % per_piece) % p.blocks;
    Piece piece;
    if (!locate(p, pi, &piece)) return;
    const int64_t slot = uniform64(slot_of(p, piece.b));
    if (slot < 0) return;
    // Columns of the identity lie behind those of the values.
    const bool values = OUT || !DELTA || slice < p.value_blocks;
    const int64_t in_slot = slot * p.slot_stride + static_cast<int64_t>(h) * p.V * p.K;
    // A piece's own place for states: [pieces, heads, value, key], transitions behind them.
    const int64_t in_ends = (pi * p.nheads + h) * p.V * p.K;
    if constexpr (!OUT) {
        // A last piece's end goes to the slot, in the launch in which the sequence's first piece needs
        // the state that was there: its place keeps that one.
        if (piece.last && !piece.first && values && p.has && p.has[piece.b]) {
            const int from = slice * VW * p.K;
            const int to = (slice + 1) * VW < p.V ? from + VW * p.K : p.V * p.K;
            for (int i = from + 4 * tid; i < to; i += 4 * kChunkThreads)
                store4<float>(p.ends, in_ends + i, state_load4(p.state, p.state_dtype, in_slot + i));
        }
        if (piece.last || (!values && piece.first)) return;
    }
    const int64_t begin = piece.begin, n_all = piece.rows;
    const int columns = values ? p.V : p.K;
    const int kg = h / p.per_group;
    const int v0 = (values ? slice : slice - p.value_blocks) * VW;  // first column of the slice
    const int wv = wave * 16 * NC;                                  // the wave's in it

    const IT* q = static_cast<const IT*>(p.q) + begin * p.q_stride + static_cast<int64_t>(kg) * p.K;
    const IT* k = static_cast<const IT*>(p.k) + begin * p.k_stride + static_cast<int64_t>(kg) * p.K;
    const IT* v = static_cast<const IT*>(p.v) + begin * p.v_stride + static_cast<int64_t>(h) * p.V;
    IT* out = static_cast<IT*>(p.out) + begin * p.out_stride + static_cast<int64_t>(h) * p.V;
    const float* decay = p.decay + begin * p.decay_stride + h;
    const void* beta = nullptr;
    if constexpr (DELTA)
        beta = static_cast<const char*>(p.beta) +
               (begin * p.beta_stride + h) * (p.beta_f32 ? 4 : static_cast<int>(ES));

    // ---- the entering state
    f32x4 S[NC][KT];
    const bool has = values && (piece.first ? p.has && p.has[piece.b] : OUT);
    // The slot is read where no other workgroup of the launch writes it: by the first launch and by
    // sequences of one piece (and, of ranges that overlap, where the last piece is past the workspace and
    // not walked). Else the state lies in `ends`: of a first piece in the last one's place, of
    // another in that of the piece before it.
    const bool of_slot = piece.first && (!OUT || piece.last || pi + piece.behind >= p.pieces);
    const int dtype = of_slot ? p.state_dtype : SSU_F32;
    const int in_size = dtype == SSU_F32 ? 4 : 2;
    const void* enter = static_cast<const char*>(p.state) + in_slot * in_size;
    if (!of_slot)
        enter = p.ends + in_ends +
                (piece.first ? piece.behind : -1) * static_cast<int64_t>(p.nheads) * p.V * p.K;
    // A lane's four keys of column tile c and key tile t, in a range that ends with the last column.
    const auto place = [&](int of_lane, int c, int t) {
        const unsigned col = v0 + wv + 16 * c + of_lane % 16, key = 16 * t + 4 * (of_lane / 16);
        return key < static_cast<unsigned>(p.K) ? col * p.K + key : kOutOfRange / 4;
    };
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[c][t][i] = !OUT && !values && 16 * t + 4 * g + i == v0 + wv + 16 * c + l16 ? 1.f : 0.f;
    if (has)
        of_dtype(dtype, [&](auto type) {
            const Rsrc from = range_of(enter, p.V * p.K * in_size);
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int t = 0; t < KT; ++t) S[c][t] = load4<decltype(type)>(from, place(lane, c, t));
        });

    // ---- what a thread moves of a chunk: its segments of q, k and v, one row's decay and beta.
    // Segment i lies QROWS (VROWS) rows behind segment i - 1, in the same columns.
    Seg<IT> qr[QSEGS], kr[QSEGS], vr[VSEGS];
    float gr = 0.f;
    unsigned br = 0;  // as loaded
    const int q_row = tid / (KP / 8), q_col = tid % (KP / 8) * 8;
    const int v_row = tid / (VW / 8), v_col = v0 + tid % (VW / 8) * 8;
    const unsigned qs = static_cast<unsigned>(p.q_stride) * ES, ks = static_cast<unsigned>(p.k_stride) * ES,
                   vs = static_cast<unsigned>(p.v_stride) * ES, os = static_cast<unsigned>(p.out_stride) * ES;
    const unsigned q_at = q_col < p.K ? q_row * qs + q_col * ES : kOutOfRange;
    const unsigned k_at = q_col < p.K ? q_row * ks + q_col * ES : kOutOfRange;
    const int v_end = values ? p.V : 0;
    const unsigned v_at = v_col < v_end ? v_row * vs + v_col * ES : kOutOfRange;
    // (Loads and stores of a chunk are the same in number for every wave and chunk, past the end too:
    // a wait for one of them would else have to be for all that went before.)
    const auto load = [&](int64_t first) {
        const int n = first < n_all ? static_cast<int>(n_all - first < C ? n_all - first : C) : 0;
        if constexpr (WIDE) {
            const Rsrc rq = range_of(q, OUT ? n * qs : 0), rk = range_of(k, n * ks),
                       rv = range_of(v, n * vs);
#pragma unroll
            for (int i = 0; i < QSEGS; ++i) {
                kr[i].load(rk, k_at + i * QROWS * ks);
                if constexpr (OUT) qr[i].load(rq, q_at + i * QROWS * qs);
            }
#pragma unroll
            for (int i = 0; i < VSEGS; ++i) vr[i].load(rv, v_at + i * VROWS * vs);
        } else {
#pragma unroll
            for (int i = 0; i < QSEGS; ++i) {
                const int row = q_row + i * QROWS;
                const int most = row < n && q_col < p.K ? 8 : 0;  // key_dim is a multiple of 8
                const int64_t at = row < n ? row : 0;
                if constexpr (OUT) qr[i].gather(q + at * p.q_stride + q_col, most);
                kr[i].gather(k + at * p.k_stride + q_col, most);
            }
#pragma unroll
            for (int i = 0; i < VSEGS; ++i) {
                const int row = v_row + i * VROWS;
                vr[i].gather(v + static_cast<int64_t>(row < n ? row : 0) * p.v_stride + v_col,
                             row < n ? v_end - v_col : 0);
            }
        }
        q += C * p.q_stride;
        k += C * p.k_stride;
        v += C * p.v_stride;
        const int64_t row = first + lane < n_all ? first + lane : n_all - 1;
        gr = decay[row * p.decay_stride];
        if constexpr (DELTA) {
            const int64_t at = row * p.beta_stride;
            if (p.beta_f32)
                br = static_cast<const unsigned*>(beta)[at];
            else
                br = static_cast<const typename Bits<IT>::type*>(beta)[at];
        }
    };
    const auto store = [&](int n) {
#pragma unroll
        for (int i = 0; i < QSEGS; ++i) {
            // 4-blocks 2 (s % 4) and the next of a block of 32: pieces 0 and 1 or 2 and 3, in their
            // first or second half.
            const int row = q_row + i * QROWS, s8 = q_col / 8;
            const int piece = s8 / 4 * 4 + s8 % 2 * 2, half = s8 % 4 / 2 * 4;
            const int lo = Shape::piece_at(row, piece) + half, hi = Shape::piece_at(row, piece + 1) + half;
            u32x4 part[NI];
            if constexpr (OUT) {
                qr[i].parts(part);
#pragma unroll
                for (int t = 0; t < NI; ++t) {
                    *reinterpret_cast<u32x2*>(&lds.q[t][row][lo]) = u32x2{part[t][0], part[t][1]};
                    *reinterpret_cast<u32x2*>(&lds.q[t][row][hi]) = u32x2{part[t][2], part[t][3]};
                }
            }
            kr[i].parts(part);
#pragma unroll
            for (int t = 0; t < NI; ++t) {
                *reinterpret_cast<u32x2*>(&lds.k[t][row][lo]) = u32x2{part[t][0], part[t][1]};
                *reinterpret_cast<u32x2*>(&lds.k[t][row][hi]) = u32x2{part[t][2], part[t][3]};
            }
        }
#pragma unroll
        for (int i = 0; i < VSEGS; ++i) {
            u32x4 part[NI];
            vr[i].parts(part);
#pragma unroll
            for (int t = 0; t < NI; ++t)
                *reinterpret_cast<u32x4*>(&lds.v[t][v_row + i * VROWS][v_col - v0]) = part[t];
        }
        if (wave == 0) {
            const float own = lane < n ? decay_of(gr) : 0.f;
            const double G = running_sum(static_cast<double>(own) * 1.4426950408889634);
            // Lane 63 has G_C: rows past the end add nothing.
            const double all = __builtin_bit_cast(double, lane63(__builtin_bit_cast(uint64_t, G)));
            if (lane < C) {
                const float hi = static_cast<float>(G);
                lds.gh[lane] = hi;
                lds.gl[lane] = static_cast<float>(G - hi);
                lds.eg[lane] = __builtin_amdgcn_exp2f(hi);
                lds.ew[lane] = __builtin_amdgcn_exp2f(static_cast<float>(all - G));
                if constexpr (DELTA) {
                    const float beta = p.beta_f32 ? __uint_as_float(br)
                                                  : widen_io<IT>(static_cast<typename Bits<IT>::type>(br));
                    lds.beta[lane] = lane < n ? beta : 0.f;
                }
            }
        }
    };

    // A lane's places in rows 16 t + l % 16, per block of 32 keys; in rows 16 t + 4 g + l % 16 / 4 read
    // transposed, per pair of key tiles.
    int at[KB], at_t[KB];
    const int trow = 4 * g + l16 / 4, tcol = (l16 & 3) * 4;
#pragma unroll
    for (int x = 0; x < KB; ++x) {
        at[x] = Shape::piece_at(l16, 4 * x + g);
        at_t[x] = Shape::piece_at(trow, 4 * x + (l16 & 3));
    }

    // ---- tile (it, jt) of the scores, and of A
    const auto scores = [&](int it, int jt) {
        const int i = 16 * it + l16, ahead = i - (16 * jt + 4 * g);  // of the lane's first column
        f32x4 s = {0.f, 0.f, 0.f, 0.f}, a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < KB; ++x) {
            u32x4 kj[NI], qi[NI], ki[NI];
#pragma unroll
            for (int t = 0; t < NI; ++t) {
                kj[t] = read16(&lds.k[t][16 * jt + l16][at[x]]);
                if constexpr (OUT) qi[t] = read16(&lds.q[t][i][at[x]]);
                if constexpr (DELTA) ki[t] = read16(&lds.k[t][i][at[x]]);
            }
            if constexpr (OUT) s = mma_parts<2>(kj, qi, s);
            if constexpr (DELTA) a = mma_parts<2>(kj, ki, a);
        }
        const float gh = lds.gh[i], gl = lds.gl[i];
        const f32x4 jh = *reinterpret_cast<const f32x4*>(&lds.gh[16 * jt + 4 * g]);
        const f32x4 jl = *reinterpret_cast<const f32x4*>(&lds.gl[16 * jt + 4 * g]);
        float beta = 0.f;
        if constexpr (DELTA) beta = lds.beta[i];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float e = __builtin_amdgcn_exp2f((gh - jh[r]) + (gl - jl[r]));
            s[r] = ahead > r - 1 ? s[r] * e : 0.f;
            if constexpr (DELTA) a[r] = ahead > r ? -beta * (a[r] * e) : 0.f;
        }
        if constexpr (OUT) {
            u32x2 part[NP];
            split4(s, part);
            const int to = Shape::p_at(i, 32 * (jt / 2) + 8 * g + 4 * (jt % 2));
#pragma unroll
            for (int t = 0; t < NP; ++t) *reinterpret_cast<u32x2*>(&lds.p[t][to]) = part[t];
        }
        if constexpr (DELTA)
            *reinterpret_cast<f32x4*>(&lds.a[Shape::a_at(it, jt) + l16 * Shape::AS + 4 * g]) = a;
    };

    // The half of the first 16 rows of P that lies above the diagonal.
    if constexpr (OUT)
        if (wave == 0)
#pragma unroll
            for (int t = 0; t < NP; ++t)
                *reinterpret_cast<u32x2*>(&lds.p[t][Shape::p_at(l16, 8 * g + 4)]) = u32x2{0, 0};

    double total = 0.;  // decay of the piece, as an exponent of 2
    load(0);
    for (int64_t first = 0; first < n_all; first += C) {
        const int n = static_cast<int>(n_all - first < C ? n_all - first : C);
        store(n);
        lds_barrier();
        load(first + C);

        // ---- scores: waves 0 and 1 take the diagonal tiles, wave 2 the one below
        if constexpr (OUT || DELTA) {
        if (wave < CT) {
            scores(wave, wave);
            if constexpr (DELTA) {
                // The diagonal block's inverse: lane l column l % 16 of (1 + A)^-1, from -A as
                // stored. All of it is read before any of it is written.
                wave_fence();
                float* a = &lds.a[Shape::a_at(wave, wave)];
                // Rows are read one ahead, and not all at once, which would take 120 registers.
                float x[16];
                f32x4 row[2][4];
                unroll<16>([&](auto index) {
                    constexpr int r = decltype(index)::value;
                    if constexpr (r < 15)
#pragma unroll
                        for (int m = 0; m <= r / 4; ++m)
                            row[(r + 1) % 2][m] = *reinterpret_cast<const f32x4*>(&a[(r + 1) * Shape::AS + 4 * m]);
                    __builtin_amdgcn_sched_barrier(0);
                    float sum[4] = {r == l16 ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int m = 0; m < r; ++m) sum[m % 4] = fmaf(row[r % 2][m / 4][m % 4], x[m], sum[m % 4]);
                    x[r] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    asm volatile("" : "+v"(x[r]));  // here, not where it is stored
                });
                wave_fence();
                // (the four lanes of a column write one value)
#pragma unroll
                for (int r = 0; r < 16; ++r) a[r * Shape::AS + l16] = x[r];
            }
        }
        if (wave == 2) scores(1, 0);
        lds_barrier();
        }

        // ---- the wave's columns
        {
            // Products with the entering state: out transposed, D[value][row]; k S, D[row][value].
            // Their operands are read one step (32 keys of q or of k) ahead: the compiler would
            // read each right before its use, and wait for LDS every time.
            f32x4 O[CT][NC], W[CT][NC];
#pragma unroll
            for (int t = 0; t < CT; ++t)
#pragma unroll
                for (int c = 0; c < NC; ++c) O[t][c] = W[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
            constexpr int STEPS = (OUT + DELTA) * KB;
            u32x4 f[2][CT][NI], sp[NC][NS];
            const auto fetch = [&](auto step) {
                constexpr int s = decltype(step)::value, x = s / (OUT + DELTA);
                constexpr bool of_k = DELTA && (!OUT || s % 2);
#pragma unroll
                for (int t = 0; t < CT; ++t)
#pragma unroll
                    for (int y = 0; y < NI; ++y)
                        f[s % 2][t][y] = read16(of_k ? &lds.k[y][16 * t + l16][at[x]]
                                                     : &lds.q[y][16 * t + l16][at[x]]);
            };
            if constexpr (STEPS > 0) fetch(std::integral_constant<int, 0>());
            unroll<STEPS>([&](auto step) {
                constexpr int s = decltype(step)::value, x = s / (OUT + DELTA);
                constexpr bool of_k = DELTA && (!OUT || s % 2);
                if constexpr (s + 1 < STEPS) fetch(std::integral_constant<int, s + 1>());
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (s % (OUT + DELTA) == 0)
#pragma unroll
                    for (int c = 0; c < NC; ++c) split8(S[c][2 * x], S[c][2 * x + 1], sp[c]);
                // Products of one place after the other: none waits for the one before it.
#pragma unroll
                for (int i = 0; i < NS; ++i)
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        constexpr int last = of_k || NI == 3 ? 2 : 1;
                        if (i + j > last) continue;
#pragma unroll
                        for (int t = 0; t < CT; ++t)
#pragma unroll
                            for (int c = 0; c < NC; ++c) {
                                if constexpr (of_k)
                                    W[t][c] = mma(f[s % 2][t][j], sp[c][i], W[t][c]);
                                else
                                    O[t][c] = mma(sp[c][i], f[s % 2][t][j], O[t][c]);
                            }
                    }
            });

            // R as an operand over the chunk's rows: v as it is, or the solution.
            constexpr int NR = DELTA ? NP : NI;
            u32x4 R[NC][TB][NR];
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                f32x4 eg, be;
                if constexpr (DELTA) {
                    eg = *reinterpret_cast<const f32x4*>(&lds.eg[16 * t + 4 * g]);
                    be = *reinterpret_cast<const f32x4*>(&lds.beta[16 * t + 4 * g]);
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    f32x4 val = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int y = 0; y < NI; ++y) {
                        const u32x2 raw = read_transposed(&lds.v[y][16 * t + trow][wv + 16 * c + tcol]);
                        float f[4];
                        Pack<__bf16>::widen(raw[0], &f[0]);
                        Pack<__bf16>::widen(raw[1], &f[2]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) val[r] = y ? val[r] + f[r] : f[r];
                        if constexpr (!DELTA && OUT) {
                            R[c][t / 2][y][t % 2 * 2] = raw[0];
                            R[c][t / 2][y][t % 2 * 2 + 1] = raw[1];
                        }
                    }
                    if constexpr (DELTA) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) val[r] = be[r] * (val[r] - eg[r] * W[t][c][r]);
                    }
                    W[t][c] = val;
                }
            }
            if constexpr (DELTA) {
                // Block by block of 16 rows: minus A below the diagonal, then the block's inverse.
#pragma unroll
                for (int t = 0; t < CT; ++t)
#pragma unroll
                    for (int u = 0; u <= t; ++u) {
                        const f32x4 a = *reinterpret_cast<const f32x4*>(
                            &lds.a[Shape::a_at(t, u) + l16 * Shape::AS + 4 * g]);
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            f32x4 d = u < t ? W[t][c] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                d = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], W[u][c][r], d, 0, 0, 0);
                            W[t][c] = d;
                        }
                    }
                if constexpr (OUT)
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int x = 0; x < TB; ++x) split8(W[2 * x][c], W[2 * x + 1][c], R[c][x]);
            }

            if constexpr (OUT) {
                // P's last part comes last; where four waves share a SIMD's registers it is read only then.
                constexpr bool LATE = Shape::waves(WIDE) == 4;
                u32x4 pf[2][TB][NP - 1], rest[2][TB];
                float pe[2];
                const auto read_p = [&](int t, int x, int part) {
                    return read16(&lds.p[part][Shape::p_at(16 * t + l16, 32 * x + 8 * g)]);
                };
                const auto fetch_p = [&](int t) {
                    pe[t % 2] = lds.eg[16 * t + l16];
#pragma unroll
                    for (int x = 0; x <= t / 2; ++x) {
#pragma unroll
                        for (int y = 0; y + 1 < NP; ++y) pf[t % 2][x][y] = read_p(t, x, y);
                        if constexpr (!LATE) rest[t % 2][x] = read_p(t, x, NP - 1);
                    }
                };
                fetch_p(0);
                unroll<CT>([&](auto tile) {
                    constexpr int t = decltype(tile)::value;
                    if constexpr (t + 1 < CT) fetch_p(t + 1);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        O[t][c] *= pe[t % 2];
#pragma unroll
                        for (int x = 0; x <= t / 2; ++x)
                            O[t][c] = mma_parts<NP - 1>(R[c][x], pf[t % 2][x], O[t][c]);
                    }
#pragma unroll
                    for (int x = 0; x <= t / 2; ++x) {
                        if constexpr (LATE) rest[t % 2][x] = read_p(t, x, NP - 1);
#pragma unroll
                        for (int c = 0; c < NC; ++c) O[t][c] = mma(R[c][x][0], rest[t % 2][x], O[t][c]);
                    }
                });
                if constexpr (WIDE) {
                    const Rsrc ro = range_of(out, n * os);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const int col = v0 + wv + 16 * c + 4 * g;
                        const unsigned at = col < p.V ? l16 * os + col * ES : kOutOfRange;
#pragma unroll
                        for (int t = 0; t < CT; ++t) {
                            float y[4];
#pragma unroll
                            for (int r = 0; r < 4; ++r) y[r] = p.scale * O[t][c][r];
                            const auto w = Raw<IT, 4>::narrow(y);
                            if constexpr (sizeof(IT) == 4)
                                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), ro,
                                                                       at + 16 * t * os, 0, 0);
                            else
                                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, w), ro,
                                                                      at + 16 * t * os, 0, 0);
                        }
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < CT; ++t) {
                        const int i = 16 * t + l16;
                        if (i >= n) continue;
                        IT* o = out + i * p.out_stride;
#pragma unroll
                        for (int c = 0; c < NC; ++c)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int col = v0 + wv + 16 * c + 4 * g + r;
                                if (col < p.V) o[col] = static_cast<IT>(p.scale * O[t][c][r]);
                            }
                    }
                }
            }

            // S = e^(G_C) S + k^T (weighted R).
            const float egc = lds.eg[C - 1];
            if constexpr (!OUT && !DELTA)
                total += static_cast<double>(lds.gh[C - 1]) + static_cast<double>(lds.gl[C - 1]);
            u32x4 wr[NC][TB][3];
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                const f32x4 w = *reinterpret_cast<const f32x4*>(&lds.ew[16 * t + 4 * g]);
#pragma unroll
                for (int c = 0; c < NC; ++c) W[t][c] *= w;
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int x = 0; x < TB; ++x) split8(W[2 * x][c], W[2 * x + 1][c], wr[c][x]);
#pragma unroll
                for (int t = 0; t < KT; ++t) S[c][t] *= egc;
            }
            // Key tiles two at a time (one of wider inputs), read ahead like the operands above.
            constexpr int KN = NI == 1 ? 2 : 1;
            u32x4 kt[2][KN][TB][NI];
            const auto fetch_k = [&](int pair) {
#pragma unroll
                for (int u = 0; u < KN; ++u)
#pragma unroll
                    for (int x = 0; x < TB; ++x)
#pragma unroll
                        for (int y = 0; y < NI; ++y) {
                            const int t = KN * pair + u, to = at_t[t / 2] + t % 2 * 4;
                            kt[pair % 2][u][x][y] =
                                join(read_transposed(&lds.k[y][32 * x + trow][to]),
                                     read_transposed(&lds.k[y][32 * x + 16 + trow][to]));
                        }
            };
            fetch_k(0);
            unroll<KT / KN>([&](auto pair) {
                constexpr int u0 = decltype(pair)::value;
                if constexpr (u0 + 1 < KT / KN) fetch_k(u0 + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < TB; ++x)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int j = 0; j < 3 - i; ++j)
#pragma unroll
                            for (int u = 0; u < KN; ++u)
#pragma unroll
                                for (int c = 0; c < NC; ++c)
                                    S[c][KN * u0 + u] =
                                        mma(kt[u0 % 2][u][x][i], wr[c][x][j], S[c][KN * u0 + u]);
            });
        }
        out += C * p.out_stride;
        lds_barrier();
    }

    // ---- the state after the last row
    if (OUT && !piece.last) return;
    int at_lane = lane;
    asm volatile("" : "+v"(at_lane));  // or the places of the entering state stay in registers until here
    const auto leave = [&](void* to, auto type) {
        typedef decltype(type) ST;
        const Rsrc r = range_of(to, columns * p.K * static_cast<int>(sizeof(ST)));
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int t = 0; t < KT; ++t) store4<ST>(r, place(at_lane, c, t), S[c][t]);
    };
    if constexpr (OUT)
        of_dtype(p.state_dtype, [&](auto type) {
            leave(static_cast<decltype(type)*>(p.state) + in_slot, type);
        });
    else
        leave(values ? p.ends + in_ends : p.moves + (pi * p.nheads + h) * p.K * p.K, float());
    if constexpr (!OUT && !DELTA)
        if (tid == 0 && slice == 0) {
            // 2^(hi + lo), lo below half a step of hi: 2^hi (1 + lo log(2)).
            const float hi = static_cast<float>(total), e = __builtin_amdgcn_exp2f(hi);
            p.sums[pi * p.nheads + h] = fmaf(e, static_cast<float>(total - hi) * layer::kLn2, e);
        }
}

// The states that enter the pieces of a sequence: ends[j] becomes M_j ends[j - 1] + ends[j] for
// every piece j >= 1 but the last, the state that enters piece j + 1.
// Without the delta rule M is a number; a workgroup takes kJoin values of one head.
constexpr int kJoin = 4 * kChunkThreads;

// The first piece of sequence b, and how many it has; by the whole wave.
__device__ __forceinline__ int64_t pieces_of(const Params& p, int64_t b, int* n) {
    const int lane = threadIdx.x & 63;
    int64_t begin, before = 0;
    for (int64_t b0 = 0; b0 < b; b0 += 64) {
        const int64_t x = b0 + lane;
        int mine = x < b ? static_cast<int>((rows_of(p, x, &begin) + p.piece - 1) / p.piece) : 0;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) mine += __shfl_xor(mine, d);
        before += mine;
    }
    *n = static_cast<int>((uniform64(rows_of(p, b, &begin)) + p.piece - 1) / p.piece);
    return uniform64(before);
}

// Whether there is a state to hand on. Row ranges that overlap (which is not allowed) can come to
// more pieces than there is room for: those past it are neither walked nor joined.
__device__ __forceinline__ bool joined(const Params& p, int64_t b, int64_t first, int n) {
    return n >= 3 && first + n <= p.pieces && slot_of(p, b) >= 0;
}

static __global__ __launch_bounds__(kChunkThreads) void join_kernel(const Params p) {
    const int64_t size = static_cast<int64_t>(p.V) * p.K, blocks = (size + kJoin - 1) / kJoin;
    const int64_t b = blockIdx.x / blocks / p.nheads;
    const int h = static_cast<int>(blockIdx.x / blocks % p.nheads);
    int n;
    const int64_t first = pieces_of(p, b, &n);
    if (!joined(p, b, first, n)) return;
    const int64_t at = blockIdx.x % blocks * kJoin + 4 * threadIdx.x;
    if (at >= size) return;  // key_dim is a multiple of 8: all four or none
    const int64_t step = p.nheads * size;
    float* e = p.ends + first * step + h * size + at;
    f32x4 S = *reinterpret_cast<const f32x4*>(e);
    f32x4 next = *reinterpret_cast<const f32x4*>(e + step);
    for (int j = 1; j + 1 < n; ++j) {
        e += step;
        const f32x4 N = next;
        if (j + 2 < n) next = *reinterpret_cast<const f32x4*>(e + step);
        S = p.sums[(first + j) * p.nheads + h] * S + N;
        *reinterpret_cast<f32x4*>(e) = S;
    }
}

// With the delta rule M is a matrix (moves holds it by columns). A workgroup takes COLS value
// columns of one head, a wave 16 or twice 16 of the keys: S goes round through LDS, as operands of
// three parts, and what the next product needs is on its way while this one runs.
template <int KP>
struct JoinShape {
    static constexpr int THREADS = KP < 128 ? KP * 4 : 512, COLS = KP == 256 ? 32 : 64;
    static constexpr int CT = COLS / 16, KB = KP / 32, TILES = KP * 4 / THREADS;
};

template <int KP>
__global__ __launch_bounds__(JoinShape<KP>::THREADS) void join_delta_kernel(const Params p) {
    constexpr int CT = JoinShape<KP>::CT, KB = JoinShape<KP>::KB, COLS = JoinShape<KP>::COLS,
                  TILES = JoinShape<KP>::TILES;
    __shared__ __attribute__((aligned(16))) unsigned short lds[2][3][KB][CT][64 * 8];
    const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int blocks = (p.V + COLS - 1) / COLS;
    const int64_t b = blockIdx.x / blocks / p.nheads;
    const int h = static_cast<int>(blockIdx.x / blocks % p.nheads);
    int n;
    const int64_t first = pieces_of(p, b, &n);
    if (!joined(p, b, first, n)) return;
    const int col = static_cast<int>(blockIdx.x % blocks) * COLS + l16;
    const int64_t step = static_cast<int64_t>(p.nheads) * p.V * p.K;
    const int64_t turn = static_cast<int64_t>(p.nheads) * p.K * p.K;
    float* e = p.ends + first * step + static_cast<int64_t>(h) * p.V * p.K;
    const float* moves = p.moves + (first * p.nheads + h) * p.K * p.K;
    // Tile u of the wave: rows 16 (TILES wave + u) of M, column c of which lies c K behind; what is past
    // the last key reads as zeros, from past the range.
    const auto row = [&](int u) { return 16 * (TILES * wave + u); };
    float m[KB][8];
    const auto load = [&](int64_t j, int u) {
        const Rsrc M = range_of(moves + j * turn, 4u * p.K * p.K);
        const int key = row(u) + l16;
        const unsigned at = key < p.K ? 4u * (4 * g * p.K + key) : kOutOfRange;
        unsigned column = 4u * p.K;
        asm volatile("" : "+s"(column));  // or every place is kept in a register from step to step
#pragma unroll
        for (int x = 0; x < KB; ++x)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m[x][i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                    M, at + (32 * x + i / 4 * 16 + i % 4) * column, 0, 0));
    };
    const auto state = [&](int64_t j, int u, int t) {
        const int v = col + 16 * t, key = row(u) + 4 * g;
        return v < p.V && key < p.K ? load4<float>(e + j * step, static_cast<int64_t>(v) * p.K + key)
                                    : f32x4{0.f, 0.f, 0.f, 0.f};
    };
    const auto pass_on = [&](int buffer, int u, const f32x4 (&S)[CT]) {
        const int tile = TILES * wave + u;
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            u32x2 part[3];
            split4(S[t], part);
#pragma unroll
            for (int i = 0; i < 3; ++i)
                *reinterpret_cast<u32x2*>(&lds[buffer][i][tile / 2][t][lane * 8 + tile % 2 * 4]) = part[i];
        }
    };
    load(1, 0);
#pragma unroll
    for (int u = 0; u < TILES; ++u) {
        f32x4 S[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) S[t] = state(0, u, t);
        pass_on(0, u, S);
    }
    for (int j = 1; j + 1 < n; ++j) {
#pragma unroll 1
        for (int u = 0; u < TILES; ++u) {
            f32x4 S[CT];
#pragma unroll
            for (int t = 0; t < CT; ++t) S[t] = state(j, u, t);
            u32x4 mp[KB][3];
#pragma unroll
            for (int x = 0; x < KB; ++x) {
                const f32x4 a = {m[x][0], m[x][1], m[x][2], m[x][3]};
                const f32x4 c = {m[x][4], m[x][5], m[x][6], m[x][7]};
                split8(a, c, mp[x]);
            }
            if (u + 1 < TILES)
                load(j, u + 1);
            else if (j + 2 < n)
                load(j + 1, 0);
            if (u == 0) __syncthreads();
#pragma unroll
            for (int x = 0; x < KB; ++x)
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    u32x4 sp[3];
#pragma unroll
                    for (int i = 0; i < 3; ++i) sp[i] = read16(&lds[(j + 1) % 2][i][x][t][lane * 8]);
                    S[t] = mma_parts<2>(mp[x], sp, S[t]);
                }
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                const int v = col + 16 * t, key = row(u) + 4 * g;
                if (v < p.V && key < p.K)
                    store4<float>(e + j * step, static_cast<int64_t>(v) * p.K + key, S[t]);
            }
            pass_on(j % 2, u, S);
        }
    }
}

template <typename IT, int KP, int NC, bool DELTA, bool WIDE>
hipError_t launch_out(Params p, hipStream_t stream) {
    p.blocks = p.value_blocks = (p.V + 64 * NC - 1) / (64 * NC);
    const int64_t grid = p.pieces * p.nheads * p.blocks;
    if (grid > INT32_MAX) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((chunk_kernel<IT, KP, NC, DELTA, WIDE, kOut>),
                       dim3(static_cast<unsigned>(grid)), dim3(kChunkThreads), 0, stream, p);
    return hipGetLastError();
}

template <typename IT, int KP, bool DELTA, bool WIDE>
hipError_t launch_ends(Params p, hipStream_t stream) {
    p.value_blocks = (p.V + 63) / 64;
    p.blocks = p.value_blocks + (DELTA ? (p.K + 63) / 64 : 0);
    const int64_t grid = p.pieces * p.nheads * p.blocks;
    const int64_t each = DELTA ? (p.V + JoinShape<KP>::COLS - 1) / JoinShape<KP>::COLS
                               : (static_cast<int64_t>(p.V) * p.K + kJoin - 1) / kJoin;
    if (grid > INT32_MAX || p.nseq * p.nheads * each > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 join(static_cast<unsigned>(p.nseq * p.nheads * each)), threads(kChunkThreads);
    hipLaunchKernelGGL((chunk_kernel<IT, KP, 1, DELTA, WIDE, kEnds>), dim3(static_cast<unsigned>(grid)),
                       threads, 0, stream, p);
    if constexpr (DELTA)
        hipLaunchKernelGGL((join_delta_kernel<KP>), join, dim3(JoinShape<KP>::THREADS), 0, stream, p);
    else
        hipLaunchKernelGGL(join_kernel, join, threads, 0, stream, p);
    return hipGetLastError();
}

template <typename IT, int KP, bool DELTA, bool WIDE>
hipError_t launch_passes(const Params& p, hipStream_t stream) {
    if (p.piece > 0) {
        const hipError_t e = launch_ends<IT, KP, DELTA, WIDE>(p, stream);
        if (e != hipSuccess) return e;
    }
    // Slices of 128 columns read q, k and P half as often; those of 64 are twice as many, and those of
    // the plain form have four waves per SIMD instead of two. From four of 64 per compute unit on the
    // wide ones gain (bf16, heads of 128 x 128; us with 64 and 128, delta rule behind: 64 of 250 rows
    // 17.2 and 23.4, 28.3 and 38.9; 512 of 64 rows 11.9 and 12.6, 16.3 and 17.1; 768 of 250 rows 33.8
    // and 38.7, 61.8 and 60.7; 1,024 of 128 rows 26.1 and 25.6, 46.7 and 38.5; 4,096 of 250 rows
    // 183 and 168, 312 and 246). Where registers are few (inputs of several parts, keys of more than
    // 128), slices of 64.
    if constexpr (std::is_same<IT, __bf16>::value && KP <= 128 && WIDE)
        if (p.piece == 0 && p.V > 64 && p.nseq * p.nheads * ((p.V + 63) / 64) >= 1024)
            return launch_out<IT, KP, 2, DELTA, WIDE>(p, stream);
    return launch_out<IT, KP, 1, DELTA, WIDE>(p, stream);
}

template <typename IT, int KP>
hipError_t launch_chunk(const Params& p, hipStream_t stream) {
    if (p.wide)
        return p.beta ? launch_passes<IT, KP, true, true>(p, stream)
                      : launch_passes<IT, KP, false, true>(p, stream);
    return p.beta ? launch_passes<IT, KP, true, false>(p, stream)
                  : launch_passes<IT, KP, false, false>(p, stream);
}

template <typename IT>
hipError_t launch_chunks(const Params& p, hipStream_t stream) {
    if (p.K <= 64) return launch_chunk<IT, 64>(p, stream);
    if (p.K <= 128) return launch_chunk<IT, 128>(p, stream);
    return launch_chunk<IT, 256>(p, stream);
}

}  // namespace attention
