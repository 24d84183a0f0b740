// layer_scan.hpp -- selective scan kernels with one decay per channel and state
// element (semantics in include/layer.h), for gfx950 (wave64).
//
// Prompts. The recurrence is serial in time and independent over channels and
// state elements, so a lane owns one channel, a wave 64 adjacent channels of one
// group and a quarter of their state elements (an eighth of 128 and 256), and a workgroup of
// four waves (eight) one piece of a sequence. Decays never leave registers; per element
// and row the work is five vector instructions, one of them an exponential at half rate:
//     a = v A;  e = 2^a;  u = v x B;  s = e s + u;  y += C s
// which is what bounds it (A is scaled by log2 e once). What the waves share passes
// through LDS a tile of kTile rows at a time: B and C, widened to fp32 and read back by
// broadcast; v and v x of every channel, of which each wave prepares its share of the
// rows; and the waves' partial y, which the wave that prepared a row sums, gates and
// stores. One barrier per tile: a tile is prepared, from inputs requested one tile earlier
// still, while the tile before it is computed.
//
// Few sequences leave most of the card idle, so long ones are then cut into
// pieces of `piece` rows: a first pass over all but a sequence's last piece finds
// the piece's own end state and sum of v (no outputs); the second pass starts each
// piece from the states joined over the pieces before it, s = exp(A sum v) s + end.
// The first pass costs about two thirds of the second. The sum of a piece's v is a chain of
// its rows over the waves and one of the waves, in fp32: it is off by at most so many half
// steps, and by far fewer as a rule.
#pragma once

#include "layer_common.hpp"

#include <type_traits>

namespace layer {

constexpr int kTile = 8;  // rows staged at a time

// Waves of a workgroup, which share a channel's state elements: with more than 16 elements
// per lane (state and A in registers) a compute unit holds too few waves.
__host__ __device__ constexpr int scan_waves(int dstate) { return dstate > 64 ? 8 : 4; }

// One piece of one sequence. `seq` < 0: no work.
struct Piece {
    int64_t seq;
    int64_t index, count; // of this piece in its sequence, and its sequence's pieces
    int64_t row;          // first packed row
    int64_t slot;
    int rows;
    bool has;             // the sequence has an initial state
};

struct ScanParams {
    void* state;
    const void* x;
    const void* z;
    const void* dt;
    const void* B;
    const void* C;
    void* out;
    const float* A;
    const float* D;
    const float* dt_bias;
    const void* cu;
    const uint8_t* has;
    const void* slots;
    int64_t nslots, slot_stride, rows, nseq, pad_slot_id;
    int64_t x_stride, z_stride, dt_stride, B_stride, C_stride, out_stride;
    int64_t piece;        // rows of a piece; 0: sequences are whole
    int64_t pieces;       // pieces there may be
    // Scratch of prompts in pieces, a sequence's pieces adjacent.
    float* ends;          // [pieces][dim][dstate]: end states; of a last piece: the entering state
    float* sums;          // [pieces][dim]: sum of v
    int32_t dim, ngroups, group_dim;
    int32_t blocks_per_group;  // channel blocks
    int32_t state_dtype, dt_f32, softplus, cu64, slot64;
    int32_t wide_bc;      // update: B and C can be read in 16-byte pieces
};

// log(1 + e^v). With u = 1 + e rounded, log1p(e) = log(u) + (e - (u - 1)) / u to first order
// in the rounding e - (u - 1), which is exact; leaving out the 1 / u is off by less than
// e 2^-24, a relative 2^-24.
__device__ __forceinline__ float softplus_fast(float v) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
    const float u = 1.f + e;
    return __builtin_amdgcn_fmed3f(v, 0.f, __builtin_inff()) +
           fmaf(__builtin_amdgcn_logf(u), kLn2, e - (u - 1.f));
}

// s 2^a, where 2^a may be out of range and the product is not: an infinite s stays infinite and
// a zero one zero for every finite a. Without a branch: one takes four registers more, which are
// a quarter of the waves where a lane has 16 elements.
__device__ __forceinline__ float scale_exp2(float s, float a) {
    const float b = __builtin_amdgcn_fmed3f(a, -4096.f, 4096.f), n = ceilf(b);
    const bool finite = fabsf(a) < __builtin_inff();
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(finite ? b - n : a) * s,
                                   finite ? static_cast<int>(n) : 0);
}

// Element i of a state of storage type `dtype`, and its store (to nearest).
__device__ __forceinline__ float state_load(const void* p, int dtype, int64_t i) {
    if (dtype == SSU_F32) return static_cast<const float*>(p)[i];
    if (dtype == SSU_F16) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
    return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}

__device__ __forceinline__ void state_store(void* p, int dtype, int64_t i, float v) {
    if (dtype == SSU_F32)
        static_cast<float*>(p)[i] = v;
    else if (dtype == SSU_F16)
        static_cast<_Float16*>(p)[i] = static_cast<_Float16>(v);
    else
        static_cast<__bf16*>(p)[i] = static_cast<__bf16>(v);
}

template <typename P>
__device__ __forceinline__ int64_t scan_slot(const P& p, int64_t b) {
    const int64_t s = p.slots ? load_index(p.slots, p.slot64, b) : b;
    return s != p.pad_slot_id && s >= 0 && s < p.nslots ? s : -1;
}

// The kernel's parameters, read from the argument segment from here on: the compiler
// otherwise loads all of them at the kernel's start, more than there are scalar registers
// beside what finding the piece takes.
typedef __attribute__((address_space(4))) const ScanParams scan_args;
__device__ __forceinline__ scan_args* fresh_args() {
    scan_args* a = (scan_args*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(a));
    return a;
}

// What a lane knows of sequence b; no rows if it is inert. The reads do not wait for each
// other: a short call is little else than dependent reads.
struct Sequence {
    int64_t begin = 0, slot = -1;
    int rows = 0, has = 0;
    __device__ __forceinline__ Sequence() {}
    __device__ __forceinline__ Sequence(const ScanParams& p, int64_t b) {
        begin = load_index(p.cu, p.cu64, b);
        const int64_t end = load_index(p.cu, p.cu64, b + 1);
        slot = scan_slot(p, b);
        has = p.has ? p.has[b] : 0;
        rows = begin >= 0 && begin <= end && end <= p.rows && slot >= 0 ? static_cast<int>(end - begin) : 0;
    }
    // Lane l's, for the whole wave.
    __device__ __forceinline__ Sequence of_lane(int l) const {
        Sequence s;
        s.begin = lane64(begin, l);
        s.slot = lane64(slot, l);
        s.rows = __builtin_amdgcn_readlane(rows, l);
        s.has = __builtin_amdgcn_readlane(has, l);
        return s;
    }
};

// Place of workgroup `id` of `n` in a list that goes from long to short work, when all
// are resident at once: workgroups reach the compute units in rounds of kUnits, and every
// second round takes its share of the list backwards, so that the shares of the units differ
// little in sum (16 prompts of mixed lengths, 1,280 workgroups: 368 us against 374). A
// bijection of [0, n).
constexpr int kUnits = 256;
__device__ __forceinline__ int fold(int id, int n) {
    const int round = id / kUnits, at = id % kUnits;
    if (round % 2 == 0 || (round + 1) * kUnits > n) return id;
    // Consecutive workgroups go to consecutive XCDs: the unit on this XCD counted from the end.
    return round * kUnits + (kUnits / ssu::kXcds - 1 - at / ssu::kXcds) * ssu::kXcds + at % ssu::kXcds;
}

// Piece `i` of the call, found by a whole wave from cu_seqlens. Whole sequences, up to 64 of
// them, go from the longest to the shortest.
__device__ __forceinline__ Piece find_piece(const ScanParams& p, int64_t i) {
    const int lane = threadIdx.x & 63;
    Piece q;
    q.seq = -1;
    q.index = 0;
    q.count = 1;
    Sequence s;
    if (p.piece == 0) {
        int64_t b = i;
        if (p.nseq <= 64) {
            Sequence mine;
            if (lane < p.nseq) mine = Sequence(p, lane);
            int rank = 0;
            for (int j = 0; j < p.nseq; ++j) {
                const int other = __builtin_amdgcn_readlane(mine.rows, j);
                rank += other > mine.rows || (other == mine.rows && j < lane);
            }
            b = __builtin_ctzll(__ballot(rank == i && lane < p.nseq) | 1ull << 63);
            s = mine.of_lane(static_cast<int>(b));
        } else {
            s = Sequence(p, b).of_lane(0);
        }
        if (s.rows > 0) q.seq = b;
        q.row = s.begin;
        q.rows = s.rows;
    } else {
        const unsigned piece_rows = static_cast<unsigned>(p.piece);
        int64_t before = 0;  // pieces of the sequences before
        for (int64_t b0 = 0; b0 < p.nseq; b0 += 64) {
            Sequence mine;
            if (b0 + lane < p.nseq) mine = Sequence(p, b0 + lane);
            const int count = static_cast<int>((static_cast<unsigned>(mine.rows) + piece_rows - 1) / piece_rows);
            int upto = count;  // of lanes 0 .. lane
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(upto, d);
                if (lane >= d) upto += o;
            }
            const unsigned long long past = __ballot(before + upto > i);
            if (past) {
                const int l = __builtin_ctzll(past);
                s = mine.of_lane(l);
                q.seq = b0 + l;
                q.count = __builtin_amdgcn_readlane(count, l);
                q.index = i - before - __builtin_amdgcn_readlane(upto, l) + q.count;
                // Decreasing cu_seqlens may name more pieces than the scratch holds.
                if (i - q.index + q.count > p.pieces) q.seq = -1;
                break;
            }
            before += __builtin_amdgcn_readlane(upto, 63);
        }
        q.row = s.begin + q.index * p.piece;
        const int64_t left = s.rows - q.index * p.piece;
        q.rows = static_cast<int>(left < p.piece ? left : p.piece);
    }
    q.seq = ssu::uniform64(q.seq);
    q.index = ssu::uniform64(q.index);
    q.count = ssu::uniform64(q.count);
    q.row = ssu::uniform64(q.row);
    q.rows = __builtin_amdgcn_readfirstlane(q.rows);
    q.slot = ssu::uniform64(s.slot);
    q.has = __builtin_amdgcn_readfirstlane(s.has) != 0;
    return q;
}

// A thread's share of a tile's inputs, as loaded: x, z and dt of the rows that its wave
// prepares, and elements of the tile's B and C.
template <typename IT, typename DT, int ROWS, int ELEMENTS>
struct Inputs {
    typename Bits<IT>::type x[ROWS], z[ROWS], bc[ELEMENTS];
    typename Bits<DT>::type dt[ROWS];
};

// What a pass over the pieces does: the first pass of prompts in pieces, or the pass that
// writes outputs and final states, without or with the gate.
enum Pass { kEnds, kPlain, kGated };

// DT: dt's type, IT or float.
template <typename IT, typename DT, int N, int PASS>
__global__ __launch_bounds__(64 * scan_waves(N)) void scan_kernel(const ScanParams args) {
    constexpr bool OUT = PASS != kEnds;
    constexpr int kWaves = scan_waves(N), kThreads = 64 * kWaves;
    constexpr int NW = N / kWaves;                 // state elements of a wave
    constexpr int kOwn = kTile / kWaves;           // rows of a tile that a wave prepares and finishes
    constexpr int kCells = kTile * 2 * N;          // elements of B and C of a tile
    constexpr int kCopies = (kCells + kThreads - 1) / kThreads;
    static_assert(kOwn >= 1 && kTile % kWaves == 0, "every wave has rows");
    typedef Inputs<IT, DT, kOwn, kCopies> In;
    typedef typename Bits<IT>::type bits;
    typedef typename Bits<DT>::type dt_bits;
    __shared__ float vs[2][2][kTile][64];                                 // v, and v x
    __shared__ __align__(16) float bs[2][kTile][2 * N];                   // B, then C
    __shared__ float ys[OUT ? 2 : 1][OUT ? kWaves : 1][OUT ? kTile : 1][64];  // partial y

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int blocks = args.blocks_per_group * args.ngroups;
    const int item = args.piece ? blockIdx.x : fold(blockIdx.x, gridDim.x);
    const int pi = item / blocks;
    const int cb = item % blocks;
    const Piece piece = find_piece(args, pi);
    const scan_args& p = *fresh_args();
    if (piece.seq < 0 || (!OUT && piece.count == 1)) return;
    const int g = cb / p.blocks_per_group;
    const int in_group = (cb % p.blocks_per_group) * 64 + lane;
    const bool active = in_group < p.group_dim;
    const int c = g * p.group_dim + (active ? in_group : p.group_dim - 1);
    const int n0 = wave * NW;
    const bool last = piece.index + 1 == piece.count;
    const bool has = piece.has;
    const int64_t at_end = static_cast<int64_t>(c) * N + n0;
    const int64_t at_state = piece.slot * p.slot_stride + at_end;
    const int64_t ends_size = static_cast<int64_t>(p.dim) * N;

    if (!OUT && last) {
        // The second pass's last piece overwrites the slot that its first piece
        // starts from: keep the entering state beside the end states.
        if (active)
#pragma unroll
            for (int i = 0; i < NW; ++i)
                p.ends[pi * ends_size + at_end + i] =
                    has ? state_load(p.state, p.state_dtype, at_state + i) : 0.f;
        return;
    }
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f;
    const float skip = OUT && p.D ? p.D[c] : 0.f;
    const bool softplus = p.softplus;
    const int rows = piece.rows;

    // This thread's elements of B and C in a tile: one column (of B, then of C), rows bc_row
    // and every kThreads / 2 N-th after it.
    static_assert(kThreads % (2 * N) == 0, "a thread stays in its column");
    constexpr int kStep = kThreads / (2 * N);
    const int bc_row = static_cast<int>(threadIdx.x) / (2 * N), bc_col = static_cast<int>(threadIdx.x) % (2 * N);
    const int64_t bc_stride = bc_col < N ? p.B_stride : p.C_stride;
    const bits* bc = static_cast<const bits*>(bc_col < N ? p.B : p.C) +
                     (piece.row + bc_row) * bc_stride + g * N + bc_col % N;
    // Requests this thread's share of the tile at row t0; each call is one tile on. Rows of x,
    // z and dt are uniform over a wave: addresses are a scalar base and the lane's channel. Rows
    // past the piece's end repeat its last one and are not used.
    const auto load = [&](int t0, In& in) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int t = t0 + wave * kOwn + j;
            const int64_t row = piece.row + (t < rows ? t : rows - 1);
            in.x[j] = (static_cast<const bits*>(p.x) + row * p.x_stride)[c];
            in.dt[j] = (static_cast<const dt_bits*>(p.dt) + row * p.dt_stride)[c];
            if (PASS == kGated) in.z[j] = (static_cast<const bits*>(p.z) + row * p.z_stride)[c];
        }
#pragma unroll
        for (int j = 0; j < kCopies; ++j)
            if (bc_row + j * kStep < kTile && t0 + bc_row + j * kStep < rows)
                in.bc[j] = bc[j * kStep * bc_stride];
        bc += kTile * bc_stride;
    };
    float total = 0.f;  // sum of v over this wave's rows
    // Prepares this thread's share of a tile for all waves, and D x and the gate of its wave's
    // rows for its own use at the tile's end.
    const auto stage = [&](int t0, const In& in, int buf, float (&dx)[kOwn], float (&gate)[kOwn]) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int t = wave * kOwn + j;
            const float d = widen_io<DT>(in.dt[j]) + bias;
            const float v = softplus ? softplus_fast(d) : d;
            const float x = widen_io<IT>(in.x[j]);
            vs[buf][0][t][lane] = v;
            vs[buf][1][t][lane] = v * x;
            if (OUT) dx[j] = skip * x;
            if (PASS == kGated) gate[j] = silu_fast(widen_io<IT>(in.z[j]));
            if (!OUT && t0 + t < rows) total += v;
        }
#pragma unroll
        for (int j = 0; j < kCopies; ++j)
            if (bc_row + j * kStep < kTile)
                bs[buf][bc_row + j * kStep][bc_col] = widen_io<IT>(in.bc[j]);
    };

    // The first tile is on its way while the state is made.
    In raw;
    float dx[kOwn], gate[kOwn];
    load(0, raw);
    float A[NW], s[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        A[i] = p.A[at_end + i] * kLog2e;
        s[i] = 0.f;
    }
    if (piece.index == 0) {
        if (has) {
            if (OUT && piece.count > 1) {
                const float* from = p.ends + (pi + piece.count - 1) * ends_size + at_end;
#pragma unroll
                for (int i = 0; i < NW; ++i) s[i] = from[i];
            } else {
#pragma unroll
                for (int i = 0; i < NW; ++i) s[i] = state_load(p.state, p.state_dtype, at_state + i);
            }
        }
    } else if (OUT) {
        // End state of piece 0 (which holds the entering state), then the others'.
        const auto join = [&](auto in_range) {
            const int64_t first = pi - piece.index;
#pragma unroll
            for (int i = 0; i < NW; ++i) s[i] = p.ends[first * ends_size + at_end + i];
#pragma unroll in_range.value && NW <= 8 ? 4 : 1
            for (int64_t k = first + 1; k < pi; ++k) {
                const float* from = p.ends + k * ends_size + at_end;
                const float sum = p.sums[k * p.dim + c];
#pragma unroll
                for (int i = 0; i < NW; ++i)
                    s[i] = in_range.value
                               ? fmaf(__builtin_amdgcn_exp2f(A[i] * sum), s[i], from[i])
                               : scale_exp2(s[i], A[i] * sum) + from[i];
            }
        };
        join(std::true_type());
        // A piece's factor may leave the range where the rows' did not: 0 times an infinite
        // state, or infinity times a zero or small one. What came of it is not finite.
        float check = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) check = fmaf(s[i], 0.f, check);
        if (__ballot(check != check)) join(std::false_type());
    }

    stage(0, raw, 0, dx, gate);
    // vmcnt(0): state and A have arrived. Left to their first use, inside the loop, the wait
    // for them would wait for every tile's inputs just requested.
    __builtin_amdgcn_s_waitcnt(0x0f70);
    if (kTile < rows) load(kTile, raw);
    lds_barrier();

    // One tile, with the next one prepared meanwhile; `which` is its half of the buffers. Two
    // copies of the body take turns, so that nothing moves between registers.
    const auto tile = [&](int t0, auto which, float (&dx)[kOwn], float (&gate)[kOwn],
                          float (&next_dx)[kOwn], float (&next_gate)[kOwn]) {
        constexpr int buf = which.value;
        if (t0 + kTile < rows) stage(t0 + kTile, raw, buf ^ 1, next_dx, next_gate);
        if (t0 + 2 * kTile < rows) load(t0 + 2 * kTile, raw);

        const auto row = [&](int t) {
            const float v = vs[buf][0][t][lane], vx = vs[buf][1][t][lane];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const float e = __builtin_amdgcn_exp2f(v * A[i]);
                s[i] = fmaf(e, s[i], vx * bs[buf][t][n0 + i]);
                if constexpr (OUT) y = fmaf(bs[buf][t][N + n0 + i], s[i], y);
            }
            if constexpr (OUT) ys[buf][wave][t][lane] = y;
        };
        if (t0 + kTile <= rows) {
#pragma unroll NW <= 8 ? kTile : NW <= 16 ? 2 : 1
            for (int t = 0; t < kTile; ++t) row(t);
        } else {
#pragma unroll 1
            for (int t = 0; t0 + t < rows; ++t) row(t);
        }
        lds_barrier();
        if constexpr (OUT) {
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const int t = wave * kOwn + j;
                float y = dx[j];
#pragma unroll
                for (int w = 0; w < kWaves; ++w) y += ys[buf][w][t][lane];
                if (PASS == kGated) y *= gate[j];
                if (t0 + t < rows && active)
                    (static_cast<IT*>(p.out) + (piece.row + t0 + t) * p.out_stride)[c] =
                        static_cast<IT>(y);
            }
        }
    };
    float other_dx[kOwn], other_gate[kOwn];
    for (int t0 = 0; t0 < rows; t0 += kTile) {
        tile(t0, std::integral_constant<int, 0>(), dx, gate, other_dx, other_gate);
        t0 += kTile;
        if (t0 >= rows) break;
        tile(t0, std::integral_constant<int, 1>(), other_dx, other_gate, dx, gate);
    }

    if constexpr (OUT) {
        if (last && active)
#pragma unroll
            for (int i = 0; i < NW; ++i) state_store(p.state, p.state_dtype, at_state + i, s[i]);
    } else {
        if (active)
#pragma unroll
            for (int i = 0; i < NW; ++i) p.ends[pi * ends_size + at_end + i] = s[i];
        float* sums = &vs[0][0][0][0];
        sums[wave * 64 + lane] = total;
        lds_barrier();
        if (wave == 0 && active) {
            float all = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) all += sums[w * 64 + lane];
            p.sums[static_cast<int64_t>(pi) * p.dim + c] = all;
        }
    }
}

// ---------------------------------------------------------------- single tokens

// Lanes share a channel's state row as 16-byte pieces: VEC elements per lane, LPR
// lanes per channel, 64 / LPR channels per wave instruction, LOADS of them in flight. A
// wave's channels lie in one group, so it reads B and C once. The state's bytes bound it:
// 512 sequences of 5,120 x 16 in fp32 (356 MB) take 67 us on states that no cache holds,
// 5.3 TB/s (a copy streams at 5.4); 76 us with loads and stores that the caches keep. One
// and four loads in flight take 74 and 66 us, rows of the same channels one after the
// other, which reads A once, 67 to 71 us.
template <typename ST, int N>
struct StepShape {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(ST));
    static constexpr int LPR = N / VEC;
    static constexpr int RPI = 64 / LPR;  // channels per instruction
};

// VEC elements of B or C, as loaded: in 16-byte pieces (or one shorter one) where alignment
// allows (WIDE), else one by one.
template <typename IT, int VEC, bool WIDE>
struct Elements {
    static constexpr int kPiece = !WIDE ? 1 : VEC * static_cast<int>(sizeof(IT)) > 16 ? 4 : VEC;
    typename Raw<IT, kPiece>::type raw[VEC / kPiece];
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const IT* p = static_cast<const IT*>(base) + at;
#pragma unroll
        for (int k = 0; k < VEC / kPiece; ++k) raw[k] = Raw<IT, kPiece>::load(p + k * kPiece);
    }
    __device__ __forceinline__ void widen(float (&f)[VEC]) const {
#pragma unroll
        for (int k = 0; k < VEC / kPiece; ++k) {
            float h[kPiece];
            Raw<IT, kPiece>::widen(raw[k], h);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) f[k * kPiece + i] = h[i];
        }
    }
};

// A load under a condition, or its conversion between two loads, would be waited for on the
// spot: all loads of a row are unconditional (an absent z or D is read as x or A and not
// used) and precede every use.
template <typename ST, typename IT, typename DT, int N, int LOADS, bool WIDE>
__global__ __launch_bounds__(256) void scan_update_kernel(const ScanParams p) {
    typedef StepShape<ST, N> Shape;
    constexpr int VEC = Shape::VEC, LPR = Shape::LPR, RPI = Shape::RPI;
    constexpr int W = VEC / Pack<ST>::kPerWord;
    typedef typename Words<W>::type words_t;
    typedef typename Bits<IT>::type bits;
    typedef typename Bits<DT>::type dt_bits;
    const int lane = threadIdx.x & 63;
    const int sub = lane % LPR;
    const int64_t wave = ssu::xcd_tile(blockIdx.x, gridDim.x) * 4 +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int blocks = p.blocks_per_group * p.ngroups;
    const int64_t b = wave / blocks;
    if (b >= p.rows) return;
    const int64_t slot = scan_slot(p, b);
    if (slot < 0) return;
    const int cb = static_cast<int>(wave % blocks);
    const int g = cb / p.blocks_per_group;
    const int first = (cb % p.blocks_per_group) * (RPI * LOADS) + lane / LPR;  // in the group
    const bits* gate = static_cast<const bits*>(p.z ? p.z : p.x);
    const int64_t gate_stride = p.z ? p.z_stride : p.x_stride;

    // Lanes past the group repeat its last channel and store nothing.
    int c[LOADS];
    bool active[LOADS];
    float A[LOADS][VEC], D[LOADS], bias[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        const int in_group = first + k * RPI;
        active[k] = in_group < p.group_dim;
        c[k] = g * p.group_dim + (active[k] ? in_group : p.group_dim - 1);
        D[k] = (p.D ? p.D : p.A)[c[k]];
        bias[k] = (p.dt_bias ? p.dt_bias : p.A)[c[k]];
#pragma unroll
        for (int i = 0; i < VEC; ++i) A[k][i] = p.A[static_cast<int64_t>(c[k]) * N + sub * VEC + i];
    }

    ST* state = static_cast<ST*>(p.state) + slot * p.slot_stride + sub * VEC;
    words_t raw[LOADS];
    bits x_in[LOADS], z_in[LOADS];
    dt_bits dt_in[LOADS];
    Elements<IT, VEC, WIDE> B_in, C_in;
#pragma unroll
    for (int k = 0; k < LOADS; ++k)
        raw[k] = __builtin_nontemporal_load(
            reinterpret_cast<const words_t*>(state + static_cast<int64_t>(c[k]) * N));
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        dt_in[k] = (static_cast<const dt_bits*>(p.dt) + b * p.dt_stride)[c[k]];
        x_in[k] = (static_cast<const bits*>(p.x) + b * p.x_stride)[c[k]];
        z_in[k] = (gate + b * gate_stride)[c[k]];
    }
    B_in.load(p.B, b * p.B_stride + g * N + sub * VEC);
    C_in.load(p.C, b * p.C_stride + g * N + sub * VEC);
    float B[VEC], C[VEC];
    B_in.widen(B);
    C_in.widen(C);
    // Stores after all arithmetic: a load's arrival is counted together with earlier stores.
    float y[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        const float x = widen_io<IT>(x_in[k]);
        const float d = widen_io<DT>(dt_in[k]) + (p.dt_bias ? bias[k] : 0.f);
        const float v = p.softplus ? softplus_fast(d) : d;
        const float vx = v * x, vl = v * kLog2e;
        float s[VEC], sum = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) Pack<ST>::widen(raw[k][i], &s[i * Pack<ST>::kPerWord]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float e = __builtin_amdgcn_exp2f(vl * A[k][i]);
            s[i] = fmaf(e, s[i], vx * B[i]);
            sum = fmaf(C[i], s[i], sum);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) raw[k][i] = Pack<ST>::narrow(&s[i * Pack<ST>::kPerWord]);
        if constexpr (LPR > 1) sum = group_sum<LPR>(sum);
        sum = fmaf(p.D ? D[k] : 0.f, x, sum);
        y[k] = sum * (p.z ? silu_fast(widen_io<IT>(z_in[k])) : 1.f);
    }
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        if (!active[k]) continue;
        __builtin_nontemporal_store(
            raw[k], reinterpret_cast<words_t*>(state + static_cast<int64_t>(c[k]) * N));
        if (sub == 0) (static_cast<IT*>(p.out) + b * p.out_stride)[c[k]] = static_cast<IT>(y[k]);
    }
}

// Channels that a wave of the update covers, for a state type's size.
constexpr int kStepLoads = 2;
__host__ inline int step_channels(int64_t dstate, int64_t state_size) {
    const int lanes = static_cast<int>(dstate * state_size / 16);
    return (64 / lanes) * kStepLoads;
}

// ---------------------------------------------------------------- the launchers

template <typename IT, typename DT>
hipError_t launch_scan_passes(const ScanParams& p, int dstate, hipStream_t stream) {
    const int64_t blocks = p.pieces * p.blocks_per_group * p.ngroups;
    if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks)), block(64 * scan_waves(dstate));
    const auto both = [&](auto n) {
        constexpr int N = decltype(n)::value;
        if (p.piece > 0)
            hipLaunchKernelGGL((scan_kernel<IT, DT, N, kEnds>), grid, block, 0, stream, p);
        if (p.z)
            hipLaunchKernelGGL((scan_kernel<IT, DT, N, kGated>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((scan_kernel<IT, DT, N, kPlain>), grid, block, 0, stream, p);
    };
    switch (dstate) {
        case 8: both(std::integral_constant<int, 8>()); break;
        case 16: both(std::integral_constant<int, 16>()); break;
        case 32: both(std::integral_constant<int, 32>()); break;
        case 64: both(std::integral_constant<int, 64>()); break;
        case 128: both(std::integral_constant<int, 128>()); break;
        case 256: both(std::integral_constant<int, 256>()); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <typename IT>
hipError_t launch_scan_varlen(const ScanParams& p, int dstate, hipStream_t stream) {
    return p.dt_f32 ? launch_scan_passes<IT, float>(p, dstate, stream)
                    : launch_scan_passes<IT, IT>(p, dstate, stream);
}

template <typename IT, typename DT, bool WIDE>
hipError_t launch_scan_step(const ScanParams& p, int dstate, hipStream_t stream) {
    const int64_t waves = p.rows * p.blocks_per_group * p.ngroups;
    if ((waves + 3) / 4 > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>((waves + 3) / 4)), block(256);
    const auto go = [&](auto n) {
        constexpr int N = decltype(n)::value, L = kStepLoads;
        if (p.state_dtype == SSU_F32)
            hipLaunchKernelGGL((scan_update_kernel<float, IT, DT, N, L, WIDE>), grid, block, 0, stream, p);
        else if (p.state_dtype == SSU_F16)
            hipLaunchKernelGGL((scan_update_kernel<_Float16, IT, DT, N, L, WIDE>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((scan_update_kernel<__bf16, IT, DT, N, L, WIDE>), grid, block, 0, stream, p);
    };
    switch (dstate) {
        case 8: go(std::integral_constant<int, 8>()); break;
        case 16: go(std::integral_constant<int, 16>()); break;
        case 32: go(std::integral_constant<int, 32>()); break;
        case 64: go(std::integral_constant<int, 64>()); break;
        case 128: go(std::integral_constant<int, 128>()); break;
        case 256: go(std::integral_constant<int, 256>()); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <typename IT>
hipError_t launch_scan_update(const ScanParams& p, int dstate, hipStream_t stream) {
    if (p.dt_f32)
        return p.wide_bc ? launch_scan_step<IT, float, true>(p, dstate, stream)
                         : launch_scan_step<IT, float, false>(p, dstate, stream);
    return p.wide_bc ? launch_scan_step<IT, IT, true>(p, dstate, stream)
                     : launch_scan_step<IT, IT, false>(p, dstate, stream);
}

// One per io dtype, each in its own translation unit.
hipError_t scan_varlen_f32(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_varlen_f16(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_varlen_bf16(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_update_f32(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_update_f16(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_update_bf16(const ScanParams& p, int dstate, hipStream_t stream);

}  // namespace layer
