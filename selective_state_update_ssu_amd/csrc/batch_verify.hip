// batch_verify.hip -- verification of drafted tokens (semantics in include/batch.h).
//
// Three launches: (scores only) the largest score, the sum of exponentials and the first
// largest token per part of each row; per sequence and tile of the vocabulary the number of
// accepted drafts and the sum of the tile's weights; per sequence the tile in which the
// drawn number falls, and the token. Rows are read once, the tile twice. Memory bounds the first
// two, latency the last. Sums of weights are fp64, so that a drawn number next to a border
// falls on the side on which the definition has it; their order is fixed.
#include "batch.h"
#include "layer_common.hpp"

namespace {

using namespace layer;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kSegs = 4;  // 16-byte segments of a thread in a tile

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
    float most;  // largest score
    int first;   // and the first token that has it, INT_MAX if there is none
    double sum;  // of exp((score - most) / temperature)
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
    double* sums;   // [nseq, ptiles, 2]: of w, of p
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

// exp(d / temperature) for d <= 0, c = log2(e) / temperature: in fp64, since a drawn number meets
// the borders of as many tokens as the vocabulary has, and each lies where the sum of all weights
// before it says (with fp32's exponential one draw in some hundreds lands on the other
// side of one, with 100,000 tokens). 2^t is 2^n e^x, |x| <= log(2) / 2, and e^x its series
// to x^10 / 10!, off by 3e-13. Minus infinity and what is below 2^-1000 gives 0.
__device__ __forceinline__ double exp_of(float d, double c) {
    const double t = static_cast<double>(d) * c;
    const double n = __builtin_rint(t);
    const double x = (t - n) * 0.69314718055994530942;
    double e = 1. / 3628800.;
    e = fma(e, x, 1. / 362880.);
    e = fma(e, x, 1. / 40320.);
    e = fma(e, x, 1. / 5040.);
    e = fma(e, x, 1. / 720.);
    e = fma(e, x, 1. / 120.);
    e = fma(e, x, 1. / 24.);
    e = fma(e, x, 1. / 6.);
    e = fma(e, x, .5);
    e = fma(e, x, 1.);
    e = fma(e, x, 1.);
    return t > -1000. ? __builtin_amdgcn_ldexp(e, static_cast<int>(n)) : 0.;
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

__device__ __forceinline__ Stats merge(Stats a, Stats b, double c) {
    if (b.most > a.most || (b.most == a.most && b.first < a.first)) {
        const Stats t = a;
        a = b;
        b = t;
    }
    // a holds the larger; where the two are equal (infinities too) the factor is 1.
    if (b.sum > 0.) a.sum += b.sum * (b.most == a.most ? 1. : exp_of(b.most - a.most, c));
    return a;
}

// ------------------------------------------------------------- statistics of scores

// A row's sequence is found from cu_seqlens (its temperature is needed).
template <typename T>
__global__ __launch_bounds__(kThreads) void stats_kernel(const VerifyParams p) {
    constexpr int E = seg_elements<T>();
    const int tile = blockIdx.x % p.tiles;
    const int64_t r = blockIdx.x / p.tiles;
    const int64_t b = count_starts(p.cu, p.cu64, p.nseq + 1, r) - 1;
    if (b < 0 || b >= p.nseq) return;
    const float temperature = p.temperature[b];
    const double c = temperature > 0.f ? inverse_of(temperature) : 0.;
    const T* row = static_cast<const T*>(p.target) + r * p.target_stride;
    const int base = tile * static_cast<int>(tile_elements(sizeof(T))) - back_of(row);
    float f[kSegs][E];
#pragma unroll
    for (int s = 0; s < kSegs; ++s)
        load_seg<T>(row, base + (s * kThreads + static_cast<int>(threadIdx.x)) * E, p.vocab, f[s],
                    -INFINITY);
    Stats mine = {-INFINITY, INT_MAX, 0.};
#pragma unroll
    for (int s = 0; s < kSegs; ++s)
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (f[s][i] > mine.most) {
                mine.most = f[s][i];
                mine.first = base + (s * kThreads + static_cast<int>(threadIdx.x)) * E + i;
            }
    if (temperature > 0.f && mine.most > -INFINITY) {
#pragma unroll
        for (int s = 0; s < kSegs; ++s)
#pragma unroll
            for (int i = 0; i < E; ++i)
                // NaN counts as minus infinity.
                mine.sum += f[s][i] == mine.most  ? 1.
                            : f[s][i] < mine.most ? exp_of(f[s][i] - mine.most, c)
                                                  : 0.;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const Stats other = {__shfl_xor(mine.most, d), __shfl_xor(mine.first, d),
                             __shfl_xor(mine.sum, d)};
        mine = merge(mine, other, c);
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

// What is known of a row before its weights are read.
struct Row {
    float most, temperature;
    int first;
    double c, sum;
};

__device__ __forceinline__ Row row_stats(const VerifyParams& p, int64_t b, int64_t r) {
    Row row = {0.f, 1.f, 0, 0., 1.};
    if (!p.temperature) return row;
    row.temperature = p.temperature[b];
    if (row.temperature > 0.f) row.c = inverse_of(row.temperature);
    Stats all = {-INFINITY, INT_MAX, 0.};
    for (int t = 0; t < p.tiles; ++t) all = merge(all, p.stats[r * p.tiles + t], row.c);
    row.most = all.most;
    row.first = all.first == INT_MAX ? 0 : all.first;
    row.sum = all.sum;
    return row;
}

// The probability of a token with this target value, not above 0 as 0.
__device__ __forceinline__ double chance(const VerifyParams& p, const Row& row, float value, int token,
                                         double inverse) {
    if (!p.temperature) return value > 0.f ? static_cast<double>(value) : 0.;
    if (!(row.temperature > 0.f)) return token == row.first ? 1. : 0.;
    if (!(row.most > -INFINITY)) return 0.;
    return (value == row.most  ? 1.
            : value < row.most ? exp_of(value - row.most, row.c)
                               : 0.) *
           inverse;
}

__device__ __forceinline__ float value_of(const void* base, int dtype, int64_t i) {
    if (dtype == SSU_F32) return static_cast<const float*>(base)[i];
    if (dtype == SSU_F16) return static_cast<float>(static_cast<const _Float16*>(base)[i]);
    return static_cast<float>(static_cast<const __bf16*>(base)[i]);
}

// The accepted drafts of a sequence, found by a whole wave: 64 drafts at a time.
template <typename T>
__device__ __forceinline__ int accepted_of(const VerifyParams& p, int64_t b, int64_t begin, int n) {
    const int lane = threadIdx.x & 63;
    for (int first = 0; first < n; first += 64) {
        const int i = first + lane;
        bool taken = false;
        if (i < n) {
            const int64_t x = load_index(p.drafts, p.draft64,
                                         b * p.draft_seq_stride + i * p.draft_step_stride);
            if (x >= 0 && x < p.vocab) {
                const int64_t r = begin + i;
                const float value =
                    static_cast<float>((static_cast<const T*>(p.target) + r * p.target_stride)[x]);
                const float q = p.probs ? value_of(p.probs, p.probs_dtype,
                                                   b * p.probs_seq_stride + i * p.probs_step_stride + x)
                                        : 1.f;
                const Row row = row_stats(p, b, r);
                const double px = chance(p, row, value, static_cast<int>(x), 1. / row.sum);
                taken = static_cast<double>(p.uniforms[b * p.uniform_stride + i]) * q < px;
            }
        }
        const unsigned long long missed = ~__ballot(taken);
        const int stop = missed ? __builtin_ctzll(missed) : 64;
        if (stop < 64) return first + stop < n ? first + stop : n;
    }
    return n;
}

// The weights of one segment of the row in question: w (what a token is drawn from) and p.
template <typename T, typename Q>
__device__ __forceinline__ void seg_weights(const VerifyParams& p, const Row& row, const T* target,
                                            const Q* probs, int64_t draft, bool rejected,
                                            double inverse, int first,
                                            double (&w)[seg_elements<T>()],
                                            double (&full)[seg_elements<T>()]) {
    constexpr int E = seg_elements<T>(), EQ = seg_elements<Q>();
    float f[E], q[E];
    load_seg<T>(target, first, p.vocab, f, p.temperature ? -INFINITY : 0.f);
    if (rejected && probs) {
        // As many elements of the other row; aligned like this one's or element by element.
        if (first >= 0 && first + E <= p.vocab && EQ <= E &&
            reinterpret_cast<uintptr_t>(probs + first) % 16 == 0) {
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
                q[i] = first + i >= 0 && first + i < p.vocab ? static_cast<float>(probs[first + i]) : 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) q[i] = rejected && first + i == draft ? 1.f : 0.f;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const bool in = first + i >= 0 && first + i < p.vocab;
        full[i] = in ? chance(p, row, f[i], first + i, inverse) : 0.;
        const double left = full[i] - static_cast<double>(q[i]);
        w[i] = left > 0. ? left : 0.;  // NaN counts as 0
    }
}

// What both later launches know of a sequence.
template <typename T, typename Q>
struct Choice {
    int64_t begin;
    int n, accepted;
    bool rejected;
    int64_t draft;
    const T* target;
    const Q* probs;
    Row row;
    double inverse;
    int back;
};

template <typename T, typename Q>
__device__ __forceinline__ bool choose(const VerifyParams& p, int64_t b, Choice<T, Q>* o) {
    if (!rows_of(p, b, &o->begin, &o->n)) return false;
    o->accepted = __builtin_amdgcn_readfirstlane(accepted_of<T>(p, b, o->begin, o->n));
    o->rejected = o->accepted < o->n;
    const int64_t r = o->begin + o->accepted;
    o->target = static_cast<const T*>(p.target) + r * p.target_stride;
    o->probs = o->rejected && p.probs ? static_cast<const Q*>(p.probs) + b * p.probs_seq_stride +
                                            o->accepted * p.probs_step_stride
                                      : nullptr;
    o->draft = o->rejected ? load_index(p.drafts, p.draft64, b * p.draft_seq_stride +
                                                                 o->accepted * p.draft_step_stride)
                           : -1;
    o->row = row_stats(p, b, r);
    o->inverse = 1. / o->row.sum;
    o->back = back_of(o->target);
    return true;
}

// -------------------------------------------------------------------- sums of weights

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}

template <typename T, typename Q>
__global__ __launch_bounds__(kThreads) void sums_kernel(const VerifyParams p) {
    constexpr int E = seg_elements<T>();
    const int tile = blockIdx.x % p.tiles;
    const int64_t b = blockIdx.x / p.tiles;
    Choice<T, Q> o;
    if (!choose(p, b, &o)) return;
    double sw = 0., sp = 0.;
#pragma unroll
    for (int s = 0; s < kSegs; ++s) {
        const int first = tile * static_cast<int>(tile_elements(sizeof(T))) - o.back +
                          (s * kThreads + static_cast<int>(threadIdx.x)) * E;
        double w[E], full[E];
        seg_weights<T, Q>(p, o.row, o.target, o.probs, o.draft, o.rejected, o.inverse, first, w, full);
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

template <typename T, typename Q>
__global__ __launch_bounds__(kThreads) void draw_kernel(const VerifyParams p) {
    constexpr int E = seg_elements<T>();
    const int64_t b = blockIdx.x;
    int32_t* tokens = p.tokens + b * (p.window + 1);
    Choice<T, Q> o;
    if (!choose(p, b, &o)) {
        for (int64_t i = threadIdx.x; i <= p.window; i += kThreads) tokens[i] = -1;
        if (threadIdx.x == 0) p.num_accepted[b] = 0;
        return;
    }
    // Every thread adds the tiles' sums in the same order.
    const double* sums = p.sums + b * p.tiles * 2;
    double total = 0.;
    for (int t = 0; t < p.tiles; ++t) total += sums[2 * t];
    const int which = total > 0. ? 0 : 1;
    if (which) {
        total = 0.;
        for (int t = 0; t < p.tiles; ++t) total += sums[2 * t + 1];
    }
    const double aim = static_cast<double>(p.uniforms[b * p.uniform_stride + p.window]) * total;
    // The tile: the first whose running sum passes the aim; where rounding (or a drawn number that
    // is not below 1) leaves none, the last with any weight.
    int tile = -1;
    double before = 0.;
    {
        double run = 0.;
        for (int t = 0; t < p.tiles; ++t) {
            const double s = sums[2 * t + which];
            if (!(s > 0.)) continue;
            tile = t;
            before = run;
            run += s;
            if (run > aim) break;
        }
    }
    __shared__ double waves[kWaves];
    __shared__ int found[kWaves], last[kWaves];
    int token = -1;
    if (tile >= 0) {
        // A thread's segments lie side by side here, so that one running sum over the threads
        // orders the tile.
        double w[kSegs][E], mine = 0.;
#pragma unroll
        for (int s = 0; s < kSegs; ++s) {
            const int first = tile * static_cast<int>(tile_elements(sizeof(T))) - o.back +
                              (static_cast<int>(threadIdx.x) * kSegs + s) * E;
            double full[E];
            seg_weights<T, Q>(p, o.row, o.target, o.probs, o.draft, o.rejected, o.inverse, first,
                              w[s], full);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (which) w[s][i] = full[i];
                mine += w[s][i];
            }
        }
        double run = mine;
        const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const double below = __shfl_up(run, d);
            if (lane >= d) run += below;
        }
        if (lane == 63) waves[wave] = run;
        __syncthreads();
        double sum = before + (run - mine);
        for (int v = 0; v < wave; ++v) sum += waves[v];
        int hit = INT_MAX, any = -1;
#pragma unroll
        for (int s = 0; s < kSegs; ++s) {
            const int first = tile * static_cast<int>(tile_elements(sizeof(T))) - o.back +
                              (static_cast<int>(threadIdx.x) * kSegs + s) * E;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (!(w[s][i] > 0.)) continue;
                sum += w[s][i];
                any = first + i;
                if (sum > aim && hit == INT_MAX) hit = first + i;
            }
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
        token = hit != INT_MAX ? hit : any;
    }
    for (int64_t i = threadIdx.x; i <= p.window; i += kThreads) {
        int32_t v = -1;
        if (i < o.accepted)
            v = static_cast<int32_t>(load_index(p.drafts, p.draft64,
                                                b * p.draft_seq_stride + i * p.draft_step_stride));
        else if (i == o.accepted)
            v = token;
        tokens[i] = v;
    }
    if (threadIdx.x == 0) p.num_accepted[b] = o.accepted + 1;
}

// ------------------------------------------------------------------------- host

constexpr int64_t kAlign = 256;
int64_t round_up(int64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Scratch for the largest number of tiles of any target type (fp32's).
int64_t stats_bytes(int64_t rows, int64_t vocab, bool scores) {
    return scores ? round_up(rows * tiles_of(vocab, 4) * static_cast<int64_t>(sizeof(Stats))) : 0;
}

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
    if (!a->workspace || !aligned(a->workspace, kAlign) ||
        a->workspace_bytes < static_cast<size_t>(ws))
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
    return static_cast<size_t>(stats_bytes(rows, vocab, scores != 0) +
                               round_up(nseq * tiles_of(vocab, 4) * 16));
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
    p.sums = reinterpret_cast<double*>(ws + stats_bytes(a->rows, a->vocab, a->temperature != nullptr));
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
