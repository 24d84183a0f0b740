// layer_scan.hpp -- selective scan kernels with one decay per channel and state
// element (semantics in include/layer.h), for gfx950 (wave64).
//
// Prompts. The recurrence is serial in time and independent over channels and
// state elements, so a lane owns one channel, a wave 64 adjacent channels of one
// group and a quarter of their state elements (an eighth of 256), and a workgroup of
// four waves (eight) one piece of a sequence. Decays never leave registers; per element and row the work
// is five vector instructions, one of them an exponential at half rate:
//     a = v A;  e = 2^a;  u = v x B;  s = e s + u;  y += C s
// which is what bounds it (A is scaled by log2 e once). B and C are the same for
// the whole wave: a first kernel widens them to fp32 in the order the waves take
// them, and the scan reads them through the scalar cache into scalar registers, the
// operands that a vector instruction takes besides its lanes' own for nothing.
// The lanes' v and v x (softplus once per row and channel) pass through LDS, a tile
// of kTile rows at a time: each wave prepares its share of the tile's rows for all, and
// later sums the waves' partial y of the same rows, gates and stores them.
//
// Few sequences leave most of the card idle, so long ones are then cut into
// pieces of `piece` rows: a first pass over all but a sequence's last piece finds
// the piece's own end state and sum of v (no outputs); the second pass starts each
// piece from the states joined over the pieces before it, s = exp(A sum v) s + end.
// The first pass costs about two thirds of the second.
#pragma once

#include "layer_common.hpp"

#include <type_traits>

namespace layer {

constexpr int kTile = 16;  // rows staged at a time

// Waves of a workgroup, which share a channel's state elements: 64 elements per lane and
// their decays would not fit the registers of four waves.
__host__ __device__ constexpr int scan_waves(int dstate) { return dstate > 128 ? 8 : 4; }

// One piece of one sequence. `seq` < 0: no work.
struct Piece {
    int32_t seq;
    int32_t index;        // of this piece in its sequence
    int32_t count;        // pieces of its sequence
    int32_t rows;
    int64_t row;          // first packed row
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
    int64_t piece;        // rows of a piece
    int64_t pieces;       // entries of the table
    // Scratch of the prompts' kernels.
    Piece* table;         // [pieces], a sequence's pieces adjacent
    float* bc;            // [rows][groups][waves][B: dstate / waves, C: dstate / waves]
    float* ends;          // [pieces][dim][dstate]: end states; of a last piece: the entering state
    float* sums;          // [pieces][dim]: sum of v
    int32_t dim, ngroups, group_dim;
    int32_t blocks_per_group;  // channel blocks
    int32_t state_dtype, dt_f32, softplus, cu64, slot64;
    int32_t wide_bc;      // update: B and C can be read in 16-byte pieces
};

// log(1 + e^v). log1p(e) = log(1 + e) e / ((1 + e) - 1) cancels the rounding of
// 1 + e (Goldberg, "What every computer scientist should know about floating-point
// arithmetic", 1991, theorem 4).
__device__ __forceinline__ float softplus_fast(float v) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(v));
    const float u = 1.f + e, d = u - 1.f;
    const float l = d == 0.f ? e : __builtin_amdgcn_logf(u) * kLn2 * (e * __builtin_amdgcn_rcpf(d));
    return fmaxf(v, 0.f) + (v != v ? v : l);
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

__device__ __forceinline__ int64_t scan_slot(const ScanParams& p, int64_t b) {
    const int64_t s = p.slots ? load_index(p.slots, p.slot64, b) : b;
    return s != p.pad_slot_id && s >= 0 && s < p.nslots ? s : -1;
}

// Reads through the scalar cache.
typedef __attribute__((address_space(4))) const float scalar_float;

// Widens B and C of every row to fp32 in the scan's order; workgroup 0 also cuts the
// sequences into pieces, in order, inert and empty ones into none.
constexpr int kPrepThreads = 256;

template <typename IT>
__global__ __launch_bounds__(kPrepThreads) void scan_prepare_kernel(const ScanParams p, int dstate) {
    if (blockIdx.x == 0) {
        __shared__ int64_t base[kPrepThreads];
        int64_t next = 0;
        for (int64_t b0 = 0; b0 < p.nseq; b0 += kPrepThreads) {
            const int64_t b = b0 + threadIdx.x;
            int64_t begin = 0, len = 0;
            if (b < p.nseq) {
                begin = load_index(p.cu, p.cu64, b);
                const int64_t end = load_index(p.cu, p.cu64, b + 1);
                if (begin >= 0 && begin <= end && end <= p.rows && scan_slot(p, b) >= 0)
                    len = end - begin;
            }
            const int64_t count = (len + p.piece - 1) / p.piece;
            base[threadIdx.x] = count;
            __syncthreads();
            for (int step = 1; step < kPrepThreads; step *= 2) {
                const int64_t add = threadIdx.x >= step ? base[threadIdx.x - step] : 0;
                __syncthreads();
                base[threadIdx.x] += add;
                __syncthreads();
            }
            // The table holds every piece of non-decreasing cu_seqlens; a sequence of any
            // others that does not fit is left out whole.
            const int64_t at = next + base[threadIdx.x] - count;
            const bool fits = at + count <= p.pieces;
            for (int64_t k = 0; k < count && at + k < p.pieces; ++k) {
                Piece q;
                q.seq = fits ? static_cast<int32_t>(b) : -1;
                q.index = static_cast<int32_t>(k);
                q.count = static_cast<int32_t>(count);
                q.rows = static_cast<int32_t>(len - k * p.piece < p.piece ? len - k * p.piece : p.piece);
                q.row = begin + k * p.piece;
                p.table[at + k] = q;
            }
            next += base[kPrepThreads - 1];
            __syncthreads();
        }
        for (int64_t i = next + threadIdx.x; i < p.pieces; i += kPrepThreads) p.table[i].seq = -1;
    }
    const int per_row = p.ngroups * dstate;
    const int waves = scan_waves(dstate), nw = dstate / waves;
    const int64_t total = p.rows * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kPrepThreads) {
        const int64_t row = i / per_row;
        const int gn = static_cast<int>(i % per_row);
        const int g = gn / dstate, n = gn % dstate;
        float* to = p.bc + ((row * p.ngroups + g) * waves + n / nw) * 2 * nw + n % nw;
        to[0] = static_cast<float>(static_cast<const IT*>(p.B)[row * p.B_stride + gn]);
        to[nw] = static_cast<float>(static_cast<const IT*>(p.C)[row * p.C_stride + gn]);
    }
}

// A lane's inputs of the rows it prepares in one tile, as loaded.
template <typename IT, int ROWS>
struct Inputs {
    typename Bits<IT>::type x[ROWS], z[ROWS];
    unsigned dt[ROWS];
};

// One pass over the pieces; OUT: the pass that writes outputs and final states.
template <typename IT, int N, bool OUT>
__global__ __launch_bounds__(64 * scan_waves(N)) void scan_kernel(const ScanParams p) {
    constexpr int kWaves = scan_waves(N);
    constexpr int NW = N / kWaves;            // state elements of a wave
    constexpr int kOwn = kTile / kWaves;      // rows of a tile that a wave prepares and finishes
    typedef Inputs<IT, kOwn> In;
    __shared__ float4 vs[2][kTile / 2][64];                  // (v, v x) of two rows
    __shared__ float4 ys[OUT ? kWaves : 1][OUT ? kTile / 4 : 1][64];  // partial y of four rows

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int blocks = p.blocks_per_group * p.ngroups;
    const int64_t pi = blockIdx.x / blocks;
    const int cb = blockIdx.x % blocks;
    const Piece piece = p.table[pi];
    if (piece.seq < 0 || (!OUT && piece.count == 1)) return;
    const int g = cb / p.blocks_per_group;
    const int in_group = (cb % p.blocks_per_group) * 64 + lane;
    const bool active = in_group < p.group_dim;
    const int c = g * p.group_dim + (active ? in_group : p.group_dim - 1);
    const int n0 = wave * NW;
    const int64_t slot = scan_slot(p, piece.seq);
    const bool last = piece.index + 1 == piece.count;
    const bool has = p.has && p.has[piece.seq];
    const int64_t at_state = slot * p.slot_stride + static_cast<int64_t>(c) * N + n0;
    const int64_t at_end = static_cast<int64_t>(c) * N + n0;
    const int64_t ends_size = static_cast<int64_t>(p.dim) * N;

    float A[NW], s[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        A[i] = p.A[static_cast<int64_t>(c) * N + n0 + i] * kLog2e;
        s[i] = 0.f;
    }
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
        for (int64_t k = pi - piece.index; k < pi; ++k) {
            const float* from = p.ends + k * ends_size + at_end;
            const float sum = p.sums[k * p.dim + c];
#pragma unroll
            for (int i = 0; i < NW; ++i)
                s[i] = fmaf(__builtin_amdgcn_exp2f(A[i] * sum), s[i], from[i]);
        }
    }

    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f;
    const float skip = OUT && p.D ? p.D[c] : 0.f;
    const int64_t row0 = piece.row;
    const int rows = piece.rows;

    // Rows are uniform over a wave: addresses are a scalar base and the lane's channel.
    const auto load = [&](int t0, In& in) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int t = t0 + wave * kOwn + j;
            const int64_t row = row0 + (t < rows ? t : rows - 1);
            typedef typename Bits<IT>::type bits;
            in.x[j] = (reinterpret_cast<const bits*>(p.x) + row * p.x_stride)[c];
            if (p.dt_f32)
                in.dt[j] = (static_cast<const unsigned*>(p.dt) + row * p.dt_stride)[c];
            else
                in.dt[j] = (reinterpret_cast<const bits*>(p.dt) + row * p.dt_stride)[c];
            if (OUT && p.z) in.z[j] = (reinterpret_cast<const bits*>(p.z) + row * p.z_stride)[c];
        }
    };
    float total = 0.f;  // sum of v over this wave's rows
    const auto stage = [&](int t0, const In& in, int buf) {
        float v[kOwn], vx[kOwn];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            float d = p.dt_f32 ? __uint_as_float(in.dt[j])
                               : widen_io<IT>(static_cast<typename Bits<IT>::type>(in.dt[j]));
            d += bias;
            if (p.softplus) d = softplus_fast(d);
            // Rows past the piece's end repeat its last one and are not used.
            const bool in_piece = t0 + wave * kOwn + j < rows;
            v[j] = d;
            vx[j] = d * widen_io<IT>(in.x[j]);
            if (!OUT && in_piece) total += d;
        }
#pragma unroll
        for (int j = 0; j < kOwn; j += 2)
            vs[buf][(wave * kOwn + j) / 2][lane] = make_float4(v[j], vx[j], v[j + 1], vx[j + 1]);
    };

    In now, next;
    load(0, now);
    stage(0, now, 0);
    if (kTile < rows) load(kTile, next);
    lds_barrier();
    scalar_float* bc = (scalar_float*)(p.bc + ((row0 * p.ngroups + g) * kWaves + wave) * 2 * NW);
    const int64_t bc_row = static_cast<int64_t>(p.ngroups) * kWaves * 2 * NW;

    for (int t0 = 0, buf = 0; t0 < rows; t0 += kTile, buf ^= 1) {
        const bool more = t0 + kTile < rows;
        if (more) stage(t0 + kTile, next, buf ^ 1);
        const In mine = now;
        now = next;
        if (t0 + 2 * kTile < rows) load(t0 + 2 * kTile, next);

        // Four rows: `full` says at compile time that none lies past the piece's end.
        const auto four = [&](int q, auto full) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            const float4 p0 = vs[buf][2 * q][lane], p1 = vs[buf][2 * q + 1][lane];
            const float v[4] = {p0.x, p0.z, p1.x, p1.z}, vx[4] = {p0.y, p0.w, p1.y, p1.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t0 + 4 * q + j;
                if (!full.value && t >= rows) break;
                scalar_float* b = bc + t * bc_row;
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const float e = __builtin_amdgcn_exp2f(v[j] * A[i]);
                    s[i] = fmaf(e, s[i], vx[j] * b[i]);
                    if constexpr (OUT) y[j] = fmaf(b[NW + i], s[i], y[j]);
                }
            }
            if constexpr (OUT) ys[wave][q][lane] = make_float4(y[0], y[1], y[2], y[3]);
        };
        if (t0 + kTile <= rows) {
#pragma unroll 1
            for (int q = 0; q < kTile / 4; ++q) four(q, std::true_type());
        } else {
#pragma unroll 1
            for (int q = 0; q < kTile / 4; ++q) four(q, std::false_type());
        }
        lds_barrier();
        if constexpr (OUT) {
            // This wave's rows: the partial sums of each.
            float y[kOwn];
            const int q = wave * kOwn / 4, first = wave * kOwn % 4;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) y[j] = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float* part = reinterpret_cast<const float*>(&ys[w][q][lane]) + first;
#pragma unroll
                for (int j = 0; j < kOwn; ++j) y[j] += part[j];
            }
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const int t = t0 + wave * kOwn + j;
                float v = fmaf(skip, widen_io<IT>(mine.x[j]), y[j]);
                if (p.z) v *= silu_fast(widen_io<IT>(mine.z[j]));
                if (t < rows && active)
                    (static_cast<IT*>(p.out) + (row0 + t) * p.out_stride)[c] = static_cast<IT>(v);
            }
            lds_barrier();
        }
    }

    if constexpr (OUT) {
        if (last && active)
#pragma unroll
            for (int i = 0; i < NW; ++i) state_store(p.state, p.state_dtype, at_state + i, s[i]);
    } else {
        if (active)
#pragma unroll
            for (int i = 0; i < NW; ++i) p.ends[pi * ends_size + at_end + i] = s[i];
        float* sums = reinterpret_cast<float*>(&vs[0][0][0]);
        sums[wave * 64 + lane] = total;
        lds_barrier();
        if (wave == 0 && active) {
            float all = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) all += sums[w * 64 + lane];
            p.sums[pi * p.dim + c] = all;
        }
    }
}

// ---------------------------------------------------------------- single tokens

// Lanes share a channel's state row as 16-byte pieces: VEC elements per lane, LPR
// lanes per channel, 64 / LPR channels per wave instruction, kLoads of them in
// flight. A wave's channels lie in one group, so it reads B and C once.
template <typename ST, int N>
struct StepShape {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(ST));
    static constexpr int LPR = N / VEC;
    static constexpr int RPI = 64 / LPR;  // channels per instruction
};

// VEC elements of B or C at p.
template <typename IT, int VEC>
__device__ __forceinline__ void load_elements(const IT* p, bool wide, float (&f)[VEC]) {
    constexpr int kPiece = VEC * static_cast<int>(sizeof(IT)) > 16 ? 4 : VEC;
    if (wide) {
#pragma unroll
        for (int k = 0; k < VEC; k += kPiece) {
            float h[kPiece];
            Raw<IT, kPiece>::widen(Raw<IT, kPiece>::load(p + k), h);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) f[k + i] = h[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = static_cast<float>(p[i]);
    }
}

template <typename ST, typename IT, int N, int LOADS>
__global__ __launch_bounds__(256) void scan_update_kernel(const ScanParams p) {
    typedef StepShape<ST, N> Shape;
    constexpr int VEC = Shape::VEC, LPR = Shape::LPR, RPI = Shape::RPI;
    constexpr int W = VEC / Pack<ST>::kPerWord;
    typedef typename Words<W>::type words_t;
    const int lane = threadIdx.x & 63;
    const int sub = lane % LPR;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * 4 +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int blocks = p.blocks_per_group * p.ngroups;
    const int64_t b = wave / blocks;
    if (b >= p.rows) return;
    const int cb = static_cast<int>(wave % blocks);
    const int64_t slot = scan_slot(p, b);
    if (slot < 0) return;
    const int g = cb / p.blocks_per_group;
    const int first = (cb % p.blocks_per_group) * (RPI * LOADS) + lane / LPR;  // in the group

    words_t raw[LOADS];
    float x[LOADS], d[LOADS], z[LOADS];
    ST* state = static_cast<ST*>(p.state) + slot * p.slot_stride + sub * VEC;
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        const int in_group = first + k * RPI;
        if (in_group >= p.group_dim) continue;
        const int c = g * p.group_dim + in_group;
        raw[k] = __builtin_nontemporal_load(
            reinterpret_cast<const words_t*>(state + static_cast<int64_t>(c) * N));
        x[k] = static_cast<float>((static_cast<const IT*>(p.x) + b * p.x_stride)[c]);
        d[k] = p.dt_f32 ? (static_cast<const float*>(p.dt) + b * p.dt_stride)[c]
                        : static_cast<float>((static_cast<const IT*>(p.dt) + b * p.dt_stride)[c]);
        if (p.z) z[k] = static_cast<float>((static_cast<const IT*>(p.z) + b * p.z_stride)[c]);
    }
    float B[VEC], C[VEC];
    load_elements<IT, VEC>(static_cast<const IT*>(p.B) + b * p.B_stride + g * N + sub * VEC,
                           p.wide_bc, B);
    load_elements<IT, VEC>(static_cast<const IT*>(p.C) + b * p.C_stride + g * N + sub * VEC,
                           p.wide_bc, C);
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        const int in_group = first + k * RPI;
        // The lanes of a channel agree here, so its sum has all of them.
        if (in_group >= p.group_dim) continue;
        const int c = g * p.group_dim + in_group;
        float v = d[k] + (p.dt_bias ? p.dt_bias[c] : 0.f);
        if (p.softplus) v = softplus_fast(v);
        const float vx = v * x[k];
        const float* A = p.A + static_cast<int64_t>(c) * N + sub * VEC;
        float s[VEC], y = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) Pack<ST>::widen(raw[k][i], &s[i * Pack<ST>::kPerWord]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float e = __builtin_amdgcn_exp2f(v * (A[i] * kLog2e));
            s[i] = fmaf(e, s[i], vx * B[i]);
            y = fmaf(C[i], s[i], y);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) raw[k][i] = Pack<ST>::narrow(&s[i * Pack<ST>::kPerWord]);
        __builtin_nontemporal_store(raw[k],
                                    reinterpret_cast<words_t*>(state + static_cast<int64_t>(c) * N));
        if constexpr (LPR > 1) y = group_sum<LPR>(y);
        if (sub == 0) {
            if (p.D) y = fmaf(p.D[c], x[k], y);
            if (p.z) y *= silu_fast(z[k]);
            (static_cast<IT*>(p.out) + b * p.out_stride)[c] = static_cast<IT>(y);
        }
    }
}

// Channels that a wave of the update covers, for a state type's size.
constexpr int kStepLoads = 2;
__host__ inline int step_channels(int64_t dstate, int64_t state_size) {
    const int lanes = static_cast<int>(dstate * state_size / 16);
    return (64 / lanes) * kStepLoads;
}

// ---------------------------------------------------------------- the launchers

template <typename IT>
hipError_t launch_scan_varlen(const ScanParams& p, int dstate, hipStream_t stream) {
    const int64_t cells = p.rows * p.ngroups * dstate;
    const int64_t want = (cells + 4 * kPrepThreads - 1) / (4 * kPrepThreads);
    const unsigned prep = static_cast<unsigned>(want < 1 ? 1 : want < 2048 ? want : 2048);
    hipLaunchKernelGGL((scan_prepare_kernel<IT>), dim3(prep), dim3(kPrepThreads), 0, stream, p,
                       dstate);
    const int64_t grid64 = p.pieces * p.blocks_per_group * p.ngroups;
    if (grid64 > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(grid64)), block(64 * scan_waves(dstate));
    const auto both = [&](auto n) {
        constexpr int N = decltype(n)::value;
        if (p.piece < p.rows)
            hipLaunchKernelGGL((scan_kernel<IT, N, false>), grid, block, 0, stream, p);
        hipLaunchKernelGGL((scan_kernel<IT, N, true>), grid, block, 0, stream, p);
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
hipError_t launch_scan_update(const ScanParams& p, int dstate, hipStream_t stream) {
    const int64_t waves = p.rows * p.blocks_per_group * p.ngroups;
    if ((waves + 3) / 4 > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>((waves + 3) / 4)), block(256);
    const auto go = [&](auto n) {
        constexpr int N = decltype(n)::value;
        if (p.state_dtype == SSU_F32)
            hipLaunchKernelGGL((scan_update_kernel<float, IT, N, kStepLoads>), grid, block, 0, stream, p);
        else if (p.state_dtype == SSU_F16)
            hipLaunchKernelGGL((scan_update_kernel<_Float16, IT, N, kStepLoads>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((scan_update_kernel<__bf16, IT, N, kStepLoads>), grid, block, 0, stream, p);
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

// One per io dtype, each in its own translation unit.
hipError_t scan_varlen_f32(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_varlen_f16(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_varlen_bf16(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_update_f32(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_update_f16(const ScanParams& p, int dstate, hipStream_t stream);
hipError_t scan_update_bf16(const ScanParams& p, int dstate, hipStream_t stream);

}  // namespace layer
