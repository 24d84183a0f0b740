// batch_verify.hip -- verification of drafted tokens (semantics in include/batch.h).
//
// From scores a first launch takes, per tile of every row, the largest score and the sum of
// exponentials (of greedy rows the first largest token). A second one sums, per tile of the row
// that a token is drawn from, its weights, and a third finds the tile in which the drawn number falls
// and the token in it. Rows are read once, but for the one that a token is drawn from. Sums of
// weights are fp64, so that a drawn number next to a border falls on the side on which the
// definition has it; their order is fixed. (One workgroup per sequence for the second and third
// launch: 84 us instead of 40 for 128 sequences of 131,072 tokens, and no faster for four.)
//
// 128 sequences of 131,072 tokens, windows of up to 4 drafts, bf16 scores: 80-82 us (42 + 31 + 11 under
// the profiler) for 134 MB of scores. The first launch takes 17 fp64 instructions per score, about half
// of its time, and its bytes the other half (vector units 61 % busy). The second has a third of that
// work: its waves wait, two per SIMD, for the dependent reads that find the row before they
// load any of it (40 % busy). 4 sequences of 32,000 tokens, probabilities in fp32: 11 us, two launches.
#include "batch.h"
#include "layer_common.hpp"

namespace {

using namespace layer;

constexpr int kThreads = 256, kWaves = kThreads / 64;   // of a tile's statistics
constexpr int kSegs = 4;                                // 16-byte segments of a thread in a tile

template <typename T>
__host__ __device__ constexpr int seg_elements() { return 16 / static_cast<int>(sizeof(T)); }
__host__ __device__ constexpr int64_t tile_elements(int64_t size) {
    return kThreads * kSegs * (16 / size);
}
// Tiles that hold a row wherever it begins in its first 16 bytes.
__host__ inline int64_t tiles_of(int64_t vocab, int64_t size) {
    const int64_t e = tile_elements(size);
    return (vocab + 16 / size - 1 + e - 1) / e;
}

struct Stats {   // of a tile of a row
    float most;  // largest score, minus infinity if there is none
    int first;   // greedy: the first token that has it, INT_MAX if there is none
    double sum;  // else: of exp((score - most) / temperature)
};

struct Row {  // what is known of a row before its weights are read
    float most, temperature;
    int first;
    double c, inverse;  // log2(e) / temperature, 1 / sum of exponentials
};

struct Choice {  // of a sequence
    int accepted, rejected;
    int64_t draft;  // the rejected one
    Row row;
};

struct VerifyParams {
    const void* target;
    const void* drafts;
    const void* probs;  // may be NULL
    const float* uniforms;
    const float* temperature;  // NULL: target holds probabilities
    const void* cu;
    int32_t* tokens;
    int32_t* num_accepted;
    Stats* stats;   // [rows, tiles]
    int32_t* owner; // [rows]: the sequence with whose temperature a row's statistics were taken, -1: none
    double* sums;   // [nseq, tiles, 2]: of w, of p
    Choice* choice; // [nseq]
    int64_t target_stride, rows, nseq, window;
    int64_t draft_seq_stride, draft_step_stride, probs_seq_stride, probs_step_stride;
    int64_t uniform_stride;
    int32_t vocab, tiles, cu64, draft64, probs_dtype;
};

// The elements of one 16-byte aligned segment of a row that lie in the row: element `first`
// of the row (negative or past the end: outside) is the segment's first.
template <typename T>
__device__ __forceinline__ void load_seg(const T* row, int first, int vocab,
                                         float (&f)[seg_elements<T>()], float outside) {
    constexpr int E = seg_elements<T>();
    if (first >= 0 && first + E <= vocab) {
        const auto raw = *reinterpret_cast<const typename Words<4>::type*>(row + first);
#pragma unroll
        for (int i = 0; i < 4; ++i) Pack<T>::widen(raw[i], &f[i * Pack<T>::kPerWord]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            f[i] = first + i >= 0 && first + i < vocab ? static_cast<float>(row[first + i]) : outside;
    }
}

// Elements of a row before its first 16-byte boundary are those of a segment that begins
// `back` elements before it.
template <typename T>
__device__ __forceinline__ int back_of(const T* row) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
}

// 2^t for t <= 0 or a little above: in fp64, since a drawn number meets the borders of as many tokens
// as the vocabulary has, and each lies where the sum of all weights before it says (with fp32's
// exponential one draw in some hundreds lands on the other side of one, with 100,000
// tokens). 2^t is 2^n 2^x, |x| <= 1/2, and (2^x - 1) / x the polynomial that meets it in the eight
// Chebyshev points of that range: 2^x is off by 2.2e-12 of itself, and is 1 for 0. n comes from
// an addition that leaves no bits behind the point. NaN and what is below -1100 gives 0.
__device__ __forceinline__ double exp2_of(double t) {
    // (Held in scalar registers: written as they are, each costs a move per product.)
    double c[8] = {0.6931471805568324,    0.24022650695888503,    0.055504109063258665,
                   0.00961812913523614,   0.0013333478473685613,  0.0001540347518652791,
                   1.5303700711328325e-05, 1.3250805518429885e-06};
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("" : "+s"(c[i]));
    constexpr double kWhole = 6755399441055744.;  // 1.5 * 2^52
    t = fmax(t, -1100.);
    const double whole = t + kWhole;
    const double x = t - (whole - kWhole);
    double e = c[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) e = fma(e, x, c[i]);
    return __builtin_amdgcn_ldexp(fma(e, x, 1.), static_cast<int>(__builtin_bit_cast(int64_t, whole)));
}

// exp((score - most) / temperature), c = log2(e) / temperature (which may be large: the
// difference comes first). Scores of infinity weigh 1 among themselves.
__device__ __forceinline__ double weight_of(float score, float most, double c) {
    if (most == INFINITY) return score == most ? 1. : 0.;
    return exp2_of((static_cast<double>(score) - most) * c);
}

__device__ __forceinline__ double inverse_of(float temperature) {
    return 1.4426950408889634 / static_cast<double>(temperature);
}

// A sequence's rows, false if it takes no part.
__device__ __forceinline__ bool rows_of(const VerifyParams& p, int64_t b, int64_t* begin, int* n) {
    const int64_t lo = ssu::uniform64(load_index(p.cu, p.cu64, b));
    const int64_t hi = ssu::uniform64(load_index(p.cu, p.cu64, b + 1));
    *begin = lo;
    *n = static_cast<int>(hi - lo - 1);
    return lo >= 0 && hi <= p.rows && lo < hi && hi - lo - 1 <= p.window;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// The sum of the lanes up to this one.
__device__ __forceinline__ double wave_scan(double v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const double below = __shfl_up(v, d);
        if (lane >= d) v += below;
    }
    return v;
}

// What a and b, sums of weights relative to their largest scores, come to.
__device__ __forceinline__ Stats merge(Stats a, Stats b, double c) {
    if (b.most > a.most || (b.most == a.most && b.first < a.first)) {
        const Stats t = a;
        a = b;
        b = t;
    }
    // a holds the larger; where the two are equal (infinities too) the factor is 1.
    if (b.sum > 0.)
        a.sum += b.sum * (b.most == a.most ? 1.
                                           : exp2_of((static_cast<double>(b.most) - a.most) * c));
    return a;
}

// ------------------------------------------------------------- statistics of scores

// A row's sequence is found from cu_seqlens (its temperature is needed), by bisection: where a range
// runs backwards it can find another one than the range's own, which is why it is noted.
template <typename T>
__global__ __launch_bounds__(kThreads) void stats_kernel(const VerifyParams p) {
    constexpr int E = seg_elements<T>();
    const int tile = blockIdx.x % p.tiles;
    const int64_t r = blockIdx.x / p.tiles;
    const T* row = static_cast<const T*>(p.target) + r * p.target_stride;
    const int base = tile * static_cast<int>(tile_elements(sizeof(T))) - back_of(row) +
                     static_cast<int>(threadIdx.x) * E;
    float f[kSegs][E];
#pragma unroll
    for (int s = 0; s < kSegs; ++s) load_seg<T>(row, base + s * kThreads * E, p.vocab, f[s], -INFINITY);
    const int64_t b = count_starts(p.cu, p.cu64, p.nseq + 1, r) - 1;
    const bool owned = b >= 0 && b < p.nseq;
    if (tile == 0 && threadIdx.x == 0) p.owner[r] = owned ? static_cast<int32_t>(b) : -1;
    if (!owned) return;
    const float temperature = p.temperature[b];
    float most = -INFINITY;  // NaN counts as minus infinity
#pragma unroll
    for (int s = 0; s < kSegs; ++s)
#pragma unroll
        for (int i = 0; i < E; ++i) most = fmaxf(most, f[s][i]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
    Stats mine = {most, INT_MAX, 0.};
    double c = 0.;
    if (!(temperature > 0.f)) {
        if (most > -INFINITY)
#pragma unroll
            for (int s = kSegs - 1; s >= 0; --s)
#pragma unroll
                for (int i = E - 1; i >= 0; --i)
                    if (f[s][i] == most) mine.first = base + s * kThreads * E + i;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) mine.first = min(mine.first, __shfl_xor(mine.first, d));
    } else if (most > -INFINITY) {
        c = inverse_of(temperature);
        if (most == INFINITY) {
#pragma unroll
            for (int s = 0; s < kSegs; ++s)
#pragma unroll
                for (int i = 0; i < E; ++i) mine.sum += f[s][i] == most ? 1. : 0.;
        } else {
            double part[4] = {0., 0., 0., 0.};
#pragma unroll
            for (int s = 0; s < kSegs; ++s)
#pragma unroll
                for (int i = 0; i < E; ++i)
                    part[i % 4] += exp2_of((static_cast<double>(f[s][i]) - most) * c);
            mine.sum = (part[0] + part[1]) + (part[2] + part[3]);
        }
        mine.sum = wave_sum(mine.sum);
    }
    __shared__ Stats waves[kWaves];
    if (threadIdx.x % 64 == 0) waves[threadIdx.x / 64] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWaves; ++w) mine = merge(mine, waves[w], c);
        p.stats[r * p.tiles + tile] = mine;
    }
}

// --------------------------------------------------------------------- acceptance

// Statistics of a row of scores, taken by kLanes neighbouring lanes that share its tiles; each gets
// the whole.
constexpr int kLanes = 8;

// The larger of two scores and the first token that has it, over the lanes.
__device__ __forceinline__ void first_largest(float& most, int& first) {
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) {
        const float other = __shfl_xor(most, d);
        const int at = __shfl_xor(first, d);
        if (other > most || (other == most && at < first)) {
            most = other;
            first = at;
        }
    }
}

__device__ __forceinline__ void complete(Row& row, float most, int first, double sum) {
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) sum += __shfl_xor(sum, d);
    row.most = most;
    row.first = first == INT_MAX ? 0 : first;
    row.inverse = 1. / sum;
}

// The same from the row itself: for rows whose statistics were taken for another sequence, which only
// happens beside a range that runs backwards.
template <typename T>
__device__ __forceinline__ void row_anew(const VerifyParams& p, int64_t r, Row& row) {
    const T* from = static_cast<const T*>(p.target) + r * p.target_stride;
    const int lane = threadIdx.x % kLanes;
    float most = -INFINITY;
    int first = INT_MAX;
    for (int64_t x = lane; x < p.vocab; x += kLanes) {
        const float score = static_cast<float>(from[x]);
        if (score > most) {
            most = score;
            first = static_cast<int>(x);
        }
    }
    first_largest(most, first);
    double sum = 0.;
    if (row.temperature > 0.f && most > -INFINITY)
        for (int64_t x = lane; x < p.vocab; x += kLanes)
            sum += weight_of(static_cast<float>(from[x]), most, row.c);
    complete(row, most, first, sum);
}

template <typename T>
__device__ __forceinline__ Row row_stats(const VerifyParams& p, int64_t b, int64_t r) {
    Row row = {0.f, 1.f, 0, 0., 1.};
    if (!p.temperature) return row;
    row.temperature = p.temperature[b];
    if (row.temperature > 0.f) row.c = inverse_of(row.temperature);
    const Stats* stats = p.stats + r * p.tiles;
    const int lane = threadIdx.x % kLanes;
    float most = -INFINITY;
    int first = INT_MAX;
    for (int t = lane; t < p.tiles; t += kLanes) {
        const Stats s = stats[t];
        if (s.most > most) {
            most = s.most;
            first = s.first;  // of equal ones the first tile's
        }
    }
    first_largest(most, first);
    double sum = 0.;
    if (row.temperature > 0.f) {
        for (int t = lane; t < p.tiles; t += kLanes) {
            const Stats s = stats[t];
            if (s.sum > 0.)
                sum += s.sum *
                       (s.most == most ? 1. : exp2_of((static_cast<double>(s.most) - most) * row.c));
        }
    }
    complete(row, most, first, sum);
    if (p.owner[r] != b) row_anew<T>(p, r, row);
    return row;
}

// The probability of a token with this target value, not above 0 as 0.
__device__ __forceinline__ double chance(const VerifyParams& p, const Row& row, float value, int token) {
    if (!p.temperature) return value > 0.f ? static_cast<double>(value) : 0.;
    if (!(row.temperature > 0.f)) return token == row.first ? 1. : 0.;
    if (!(row.most > -INFINITY)) return 0.;
    return weight_of(value, row.most, row.c) * row.inverse;
}

__device__ __forceinline__ float value_of(const void* base, int dtype, int64_t i) {
    if (dtype == SSU_F32) return static_cast<const float*>(base)[i];
    if (dtype == SSU_F16) return static_cast<float>(static_cast<const _Float16*>(base)[i]);
    return static_cast<float>(static_cast<const __bf16*>(base)[i]);
}

// How many drafts of a sequence are accepted and what is known of the row that follows, found by a
// whole wave: kLanes lanes a row, as many rows at a time as it has room for.
template <typename T>
__device__ __forceinline__ Choice choice_of(const VerifyParams& p, int64_t b, int64_t begin, int n) {
    const int lane = threadIdx.x & 63;
    for (int base = 0;; base += 64 / kLanes) {
        const int i = base + lane / kLanes;
        bool taken = false;
        Choice c = {i, i < n, -1, {0.f, 1.f, 0, 0., 1.}};
        if (i <= n) {
            const int64_t r = begin + i;
            const bool draft = i < n;
            if (draft)
                c.draft = load_index(p.drafts, p.draft64, b * p.draft_seq_stride + i * p.draft_step_stride);
            const int64_t x = c.draft;
            const bool token = x >= 0 && x < p.vocab;
            float value = 0.f, q = 1.f;
            double u = 0.;
            if (token) {
                value = static_cast<float>((static_cast<const T*>(p.target) + r * p.target_stride)[x]);
                if (p.probs)
                    q = value_of(p.probs, p.probs_dtype,
                                 b * p.probs_seq_stride + i * p.probs_step_stride + x);
                if (q < 0.f) q = 0.f;  // (NaN stays, and rejects)
                u = static_cast<double>(p.uniforms[b * p.uniform_stride + i]);
            }
            c.row = row_stats<T>(p, b, r);
            taken = token && u * q < chance(p, c.row, value, static_cast<int>(x));
        }
        const unsigned long long missed = ~__ballot(taken);
        if (!missed) continue;  // more rows than these (one past the drafts is never taken)
        const int from = __builtin_ctzll(missed);
        Choice o;
        o.accepted = __shfl(c.accepted, from);
        o.rejected = __shfl(c.rejected, from);
        o.draft = __shfl(c.draft, from);
        o.row.most = __shfl(c.row.most, from);
        o.row.temperature = __shfl(c.row.temperature, from);
        o.row.first = __shfl(c.row.first, from);
        o.row.c = __shfl(c.row.c, from);
        o.row.inverse = __shfl(c.row.inverse, from);
        return o;
    }
}

// A sequence's row that the next token is drawn from.
template <typename T, typename Q>
struct Draw {
    const T* target;
    const Q* probs;  // NULL: q is one at the draft, or there is no rejected draft
    int64_t draft;   // -1: none was rejected
    Row row;

    // One segment's values of both rows; what lies outside the vocabulary weighs nothing.
    __device__ __forceinline__ void load(const VerifyParams& p, int first, float (&f)[seg_elements<T>()],
                                         float (&q)[seg_elements<T>()]) const {
        constexpr int E = seg_elements<T>(), EQ = seg_elements<Q>();
        load_seg<T>(target, first, p.vocab, f, p.temperature ? -INFINITY : 0.f);
        if (probs && first >= 0 && first + E <= p.vocab && EQ <= E &&
            reinterpret_cast<uintptr_t>(probs + first) % 16 == 0) {
            // As many elements of the other row where it is aligned like this one.
#pragma unroll
            for (int k = 0; k < E / EQ || k < 1; ++k) {
                const auto raw = *reinterpret_cast<const typename Words<4>::type*>(probs + first + k * EQ);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (k * EQ + i * Pack<Q>::kPerWord < E)
                        Pack<Q>::widen(raw[i], &q[k * EQ + i * Pack<Q>::kPerWord]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                q[i] = probs ? (first + i >= 0 && first + i < p.vocab ? static_cast<float>(probs[first + i])
                                                                      : 0.f)
                             : (draft >= 0 && first + i == draft ? 1.f : 0.f);
        }
    }
    // Their weights: w (what the token is drawn from) and p. What lies outside the vocabulary has
    // come as minus infinity (of probabilities: 0).
    __device__ __forceinline__ void weigh(const VerifyParams& p, const float (&f)[seg_elements<T>()],
                                          const float (&q)[seg_elements<T>()],
                                          double (&w)[seg_elements<T>()],
                                          double (&full)[seg_elements<T>()]) const {
        constexpr int E = seg_elements<T>();
        if (!p.temperature) {
#pragma unroll
            for (int i = 0; i < E; ++i) full[i] = f[i] > 0.f ? static_cast<double>(f[i]) : 0.;
        } else if (!(row.most > -INFINITY)) {
#pragma unroll
            for (int i = 0; i < E; ++i) full[i] = 0.;
        } else if (row.most == INFINITY) {
#pragma unroll
            for (int i = 0; i < E; ++i) full[i] = f[i] == INFINITY ? row.inverse : 0.;
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                full[i] = exp2_of((static_cast<double>(f[i]) - row.most) * row.c) * row.inverse;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const double left = full[i] - static_cast<double>(q[i] < 0.f ? 0.f : q[i]);
            w[i] = left > 0. ? left : 0.;  // of NaN: 0
        }
    }
};

template <typename T, typename Q>
__device__ __forceinline__ Draw<T, Q> draw_of(const VerifyParams& p, int64_t b, int64_t begin,
                                              const Choice& c) {
    Draw<T, Q> o;
    o.target = static_cast<const T*>(p.target) + (begin + c.accepted) * p.target_stride;
    o.probs = c.rejected && p.probs ? static_cast<const Q*>(p.probs) + b * p.probs_seq_stride +
                                          c.accepted * p.probs_step_stride
                                    : nullptr;
    o.draft = c.rejected ? c.draft : -1;
    o.row = c.row;
    return o;
}

// A greedy row has one token.
__device__ __forceinline__ bool greedy(const VerifyParams& p, const Row& row) {
    return p.temperature && !(row.temperature > 0.f);
}

// -------------------------------------------------------------------- sums of weights

template <typename T, typename Q>
__global__ __launch_bounds__(kThreads) void sums_kernel(const VerifyParams p) {
    constexpr int E = seg_elements<T>();
    const int tile = blockIdx.x % p.tiles;
    const int64_t b = blockIdx.x / p.tiles;
    int64_t begin;
    int n;
    if (!rows_of(p, b, &begin, &n)) return;
    Choice c = choice_of<T>(p, b, begin, n);
    c.accepted = __builtin_amdgcn_readfirstlane(c.accepted);
    c.rejected = __builtin_amdgcn_readfirstlane(c.rejected);
    if (tile == 0 && threadIdx.x == 0) p.choice[b] = c;
    if (greedy(p, c.row)) return;
    const Draw<T, Q> o = draw_of<T, Q>(p, b, begin, c);
    const int base = tile * static_cast<int>(tile_elements(sizeof(T))) - back_of(o.target) +
                     static_cast<int>(threadIdx.x) * E;
    double sw = 0., sp = 0.;
    float f[kSegs][E], q[kSegs][E];
#pragma unroll
    for (int s = 0; s < kSegs; ++s) o.load(p, base + s * kThreads * E, f[s], q[s]);
#pragma unroll
    for (int s = 0; s < kSegs; ++s) {
        double w[E], full[E];
        o.weigh(p, f[s], q[s], w, full);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            sw += w[i];
            sp += full[i];
        }
    }
    sw = wave_sum(sw);
    sp = wave_sum(sp);
    __shared__ double waves[kWaves][2];
    if (threadIdx.x % 64 == 0) {
        waves[threadIdx.x / 64][0] = sw;
        waves[threadIdx.x / 64][1] = sp;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double all = 0.;
        for (int w = 0; w < kWaves; ++w) all += waves[w][threadIdx.x];
        p.sums[(b * p.tiles + tile) * 2 + threadIdx.x] = all;
    }
}

// ----------------------------------------------------------------------- the token

// The token of a sequence that the drawn number falls to, -1 if none has any weight.
template <typename T, typename Q>
__device__ __forceinline__ int token_of(const VerifyParams& p, int64_t b, int64_t begin,
                                        const Choice& c) {
    constexpr int E = seg_elements<T>();
    const Draw<T, Q> o = draw_of<T, Q>(p, b, begin, c);
    // Every wave takes the tiles' sums, 64 at a time.
    const double* sums = p.sums + b * p.tiles * 2;
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    double total[2] = {0., 0.};
    for (int t = 0; t < p.tiles; t += 64) {
        const bool in = t + lane < p.tiles;
        total[0] += wave_sum(in ? sums[2 * (t + lane)] : 0.);
        total[1] += wave_sum(in ? sums[2 * (t + lane) + 1] : 0.);
    }
    const int which = total[0] > 0. ? 0 : 1;
    const double aim = static_cast<double>(p.uniforms[b * p.uniform_stride + p.window]) * total[which];
    // The tile: the first whose running sum passes the aim; where rounding (or a drawn number that
    // is not below 1) leaves none, the last with any weight.
    int tile = -1;
    double before = 0., run = 0.;
    for (int t = 0; t < p.tiles; t += 64) {
        const double s = t + lane < p.tiles ? sums[2 * (t + lane) + which] : 0.;
        const double upto = run + wave_scan(s);
        const unsigned long long any = __ballot(s > 0.), past = __ballot(s > 0. && upto > aim);
        if (any) {
            const int at = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(any);
            tile = t + at;
            before = __shfl(upto - s, at);
        }
        if (past) break;
        run = __shfl(upto, 63);
    }
    if (tile < 0) return -1;
    // A thread's segments lie side by side here, so that one running sum over the threads orders the
    // tile.
    const int base = tile * static_cast<int>(tile_elements(sizeof(T))) - back_of(o.target) +
                     static_cast<int>(threadIdx.x) * (kSegs * E);
    double w[kSegs][E], own = 0.;
    {
        float f[kSegs][E], q[kSegs][E];
#pragma unroll
        for (int s = 0; s < kSegs; ++s) o.load(p, base + s * E, f[s], q[s]);
#pragma unroll
        for (int s = 0; s < kSegs; ++s) {
            double full[E];
            o.weigh(p, f[s], q[s], w[s], full);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (which) w[s][i] = full[i];
                own += w[s][i];
            }
        }
    }
    __shared__ double waves[kWaves];
    __shared__ int found[kWaves], last[kWaves];
    double sum = wave_scan(own);
    if (lane == 63) waves[wave] = sum;
    __syncthreads();
    sum = before + (sum - own);
    for (int v = 0; v < wave; ++v) sum += waves[v];
    int hit = INT_MAX, any = -1;
#pragma unroll
    for (int s = 0; s < kSegs; ++s)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (!(w[s][i] > 0.)) continue;
            sum += w[s][i];
            any = base + s * E + i;
            if (sum > aim && hit == INT_MAX) hit = any;
        }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        hit = min(hit, __shfl_xor(hit, d));
        any = max(any, __shfl_xor(any, d));
    }
    if (lane == 0) {
        found[wave] = hit;
        last[wave] = any;
    }
    __syncthreads();
    hit = INT_MAX, any = -1;
    for (int v = 0; v < kWaves; ++v) {
        hit = min(hit, found[v]);
        any = max(any, last[v]);
    }
    return hit != INT_MAX ? hit : any;
}

template <typename T, typename Q>
__global__ __launch_bounds__(kThreads) void draw_kernel(const VerifyParams p) {
    const int64_t b = blockIdx.x;
    int32_t* tokens = p.tokens + b * (p.window + 1);
    int64_t begin;
    int n;
    if (!rows_of(p, b, &begin, &n)) {
        for (int64_t i = threadIdx.x; i <= p.window; i += kThreads) tokens[i] = -1;
        if (threadIdx.x == 0) p.num_accepted[b] = 0;
        return;
    }
    const Choice c = p.choice[b];
    const int token = greedy(p, c.row) ? c.row.first : token_of<T, Q>(p, b, begin, c);
    for (int64_t i = threadIdx.x; i <= p.window; i += kThreads) {
        int32_t v = -1;
        if (i < c.accepted)
            v = static_cast<int32_t>(load_index(p.drafts, p.draft64,
                                                b * p.draft_seq_stride + i * p.draft_step_stride));
        else if (i == c.accepted)
            v = token;
        tokens[i] = v;
    }
    if (threadIdx.x == 0) p.num_accepted[b] = c.accepted + 1;
}

// ------------------------------------------------------------------------- host

constexpr int64_t kAlign = 256;
int64_t round_up(int64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Scratch for the largest number of tiles of any target type (fp32's).
int64_t stats_bytes(int64_t rows, int64_t vocab, bool scores) {
    return scores ? round_up(rows * tiles_of(vocab, 4) * static_cast<int64_t>(sizeof(Stats))) : 0;
}
int64_t owner_bytes(int64_t rows, bool scores) { return scores ? round_up(rows * 4) : 0; }
int64_t sums_bytes(int64_t nseq, int64_t vocab) { return round_up(nseq * tiles_of(vocab, 4) * 16); }

int check(const ssu_verify_args* a) {
    using ssu::report;
    constexpr int kBad = SSU_ERR_INVALID_ARGUMENT;
    if (!a) return report(kBad, "args must not be NULL");
    if (a->struct_size != sizeof(ssu_verify_args))
        return report(kBad, "struct_size %u != sizeof(ssu_verify_args) %zu (header mismatch)",
                      a->struct_size, sizeof(ssu_verify_args));
    if (a->reserved != 0) return report(kBad, "reserved must be 0");
    if (!is_dtype(a->target_dtype) || (a->draft_probs && !is_dtype(a->probs_dtype)))
        return report(kBad, "target_dtype %d or probs_dtype %d is not an ssu_dtype", a->target_dtype,
                      a->probs_dtype);
    if (!is_index(a->cu_dtype) || !is_index(a->draft_dtype))
        return report(kBad, "cu_dtype %d or draft_dtype %d is not an ssu_index_dtype", a->cu_dtype,
                      a->draft_dtype);
    if (a->rows < 0 || a->vocab < 1 || a->nseq < 0 || a->window < 0)
        return report(kBad, "sizes must be positive (rows %lld, vocab %lld, nseq %lld, window %lld)",
                      (long long)a->rows, (long long)a->vocab, (long long)a->nseq,
                      (long long)a->window);
    if (a->vocab > INT32_MAX - (1 << 20) || a->window >= (1 << 20) || a->rows > INT32_MAX ||
        a->nseq > INT32_MAX)
        return report(SSU_ERR_UNSUPPORTED,
                      "vocab must be below 2^31 - 2^20, window below 2^20, rows and nseq below 2^31");
    if (a->target_stride < 0 || a->draft_seq_stride < 0 || a->draft_step_stride < 0 ||
        a->probs_seq_stride < 0 || a->probs_step_stride < 0 || a->uniform_stride < 0)
        return report(kBad, "strides must be >= 0");
    if (a->nseq == 0) return SSU_OK;
    const int64_t tsz = size_of(a->target_dtype), psz = size_of(a->probs_dtype),
                  cu = a->cu_dtype == SSU_I64 ? 8 : 4, dsz = a->draft_dtype == SSU_I64 ? 8 : 4;
    const int64_t w = a->window, ws = static_cast<int64_t>(ssu_verify_workspace_bytes(
                                     a->rows, a->nseq, a->vocab, a->temperature != nullptr));
    const struct { const char* name; int64_t align; Rows rows; bool optional; } in[] = {
        {"target", tsz, Rows(a->target, a->rows, a->target_stride, a->vocab, tsz), a->rows == 0},
        {"drafts", dsz,
         Rows(a->drafts, w ? ((a->nseq - 1) * a->draft_seq_stride + (w - 1) * a->draft_step_stride + 1) * dsz : 0),
         w == 0},
        {"draft_probs", psz,
         Rows(a->draft_probs, w ? ((a->nseq - 1) * a->probs_seq_stride + (w - 1) * a->probs_step_stride + a->vocab) * psz : 0),
         true},
        {"uniforms", 4, Rows(a->uniforms, a->nseq, a->uniform_stride, w + 1, 4), false},
        {"temperature", 4, Rows(a->temperature, a->nseq * 4), true},
        {"cu_seqlens", cu, Rows(a->cu_seqlens, (a->nseq + 1) * cu), false},
    };
    for (const auto& x : in) {
        if (!x.rows.p && !x.optional) return report(kBad, "%s must not be NULL", x.name);
        if (!aligned(x.rows.p, x.align))
            return report(kBad, "%s must be aligned to its dtype", x.name);
    }
    if (!a->tokens || !a->num_accepted)
        return report(kBad, "tokens and num_accepted must not be NULL");
    if (!aligned(a->tokens, 4) || !aligned(a->num_accepted, 4))
        return report(kBad, "tokens and num_accepted must be aligned to their dtype");
    if (ws > 0 && (!a->workspace || !aligned(a->workspace, kAlign) ||
                   a->workspace_bytes < static_cast<size_t>(ws)))
        return report(kBad, "workspace must be 256-byte aligned and hold %lld bytes (got %zu)",
                      (long long)ws, a->workspace_bytes);
    const struct { const char* name; Rows rows; } written[] = {
        {"tokens", Rows(a->tokens, a->nseq * (w + 1) * 4)},
        {"num_accepted", Rows(a->num_accepted, a->nseq * 4)},
        {"workspace", Rows(a->workspace, ws)}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& x : in)
            if (overlap(written[i].rows, x.rows))
                return report(kBad, "%s overlaps %s", written[i].name, x.name);
        for (int j = 0; j < i; ++j)
            if (overlap(written[i].rows, written[j].rows))
                return report(kBad, "%s overlaps %s", written[i].name, written[j].name);
    }
    if (a->rows * tiles_of(a->vocab, tsz) > INT32_MAX || a->nseq * tiles_of(a->vocab, tsz) > INT32_MAX)
        return report(SSU_ERR_UNSUPPORTED, "too many rows of this vocabulary for one call");
    return SSU_OK;
}

template <typename T, typename Q>
int launch(const VerifyParams& p, hipStream_t stream) {
    const char* entry = "ssu_verify_drafts";
    const dim3 threads(kThreads);
    if (p.temperature && p.rows > 0) {
        hipLaunchKernelGGL((stats_kernel<T>), dim3(static_cast<unsigned>(p.rows * p.tiles)), threads,
                           0, stream, p);
        if (int rc = launched(entry)) return rc;
    }
    hipLaunchKernelGGL((sums_kernel<T, Q>), dim3(static_cast<unsigned>(p.nseq * p.tiles)), threads, 0,
                       stream, p);
    if (int rc = launched(entry)) return rc;
    hipLaunchKernelGGL((draw_kernel<T, Q>), dim3(static_cast<unsigned>(p.nseq)), threads, 0, stream, p);
    return launched(entry);
}

template <typename T>
int launch_probs(const VerifyParams& p, hipStream_t stream) {
    if (!p.probs || p.probs_dtype == SSU_F32) return launch<T, float>(p, stream);
    if (p.probs_dtype == SSU_F16) return launch<T, _Float16>(p, stream);
    return launch<T, __bf16>(p, stream);
}

}  // namespace

extern "C" {

size_t ssu_verify_workspace_bytes(int64_t rows, int64_t nseq, int64_t vocab, int32_t scores) {
    if (rows < 0 || nseq < 0 || vocab < 1) return 0;
    return static_cast<size_t>(stats_bytes(rows, vocab, scores != 0) + owner_bytes(rows, scores != 0) +
                               sums_bytes(nseq, vocab) + nseq * static_cast<int64_t>(sizeof(Choice)));
}

int ssu_verify_drafts(const ssu_verify_args* a, void* stream) {
    if (int rc = check(a)) return rc;
    if (a->nseq == 0) return ssu::report_ok();
    VerifyParams p{};
    p.target = a->target;
    p.drafts = a->drafts;
    p.probs = a->draft_probs;
    p.uniforms = a->uniforms;
    p.temperature = a->temperature;
    p.cu = a->cu_seqlens;
    p.tokens = a->tokens;
    p.num_accepted = a->num_accepted;
    char* ws = static_cast<char*>(a->workspace);
    p.stats = reinterpret_cast<Stats*>(ws);
    ws += stats_bytes(a->rows, a->vocab, a->temperature != nullptr);
    p.owner = reinterpret_cast<int32_t*>(ws);
    ws += owner_bytes(a->rows, a->temperature != nullptr);
    p.sums = reinterpret_cast<double*>(ws);
    p.choice = reinterpret_cast<Choice*>(ws + sums_bytes(a->nseq, a->vocab));
    p.target_stride = a->target_stride;
    p.rows = a->rows;
    p.nseq = a->nseq;
    p.window = a->window;
    p.draft_seq_stride = a->draft_seq_stride;
    p.draft_step_stride = a->draft_step_stride;
    p.probs_seq_stride = a->probs_seq_stride;
    p.probs_step_stride = a->probs_step_stride;
    p.uniform_stride = a->uniform_stride;
    p.vocab = static_cast<int32_t>(a->vocab);
    p.tiles = static_cast<int32_t>(tiles_of(a->vocab, size_of(a->target_dtype)));
    p.cu64 = a->cu_dtype == SSU_I64;
    p.draft64 = a->draft_dtype == SSU_I64;
    p.probs_dtype = a->probs_dtype;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->target_dtype == SSU_F32) return launch_probs<float>(p, st);
    if (a->target_dtype == SSU_F16) return launch_probs<_Float16>(p, st);
    return launch_probs<__bf16>(p, st);
}

}  // extern "C"
