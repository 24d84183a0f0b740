// layer_conv.hip -- short causal depthwise convolution over packed prompts and for
// single tokens (semantics in include/layer.h).
//
// Both kernels give a lane VEC adjacent channels (16 bytes of a row when
// alignment allows, else one channel) and hold their width taps, bias and the
// last width - 1 inputs in fp32 registers, so each input is read and each output
// written once. Memory bounds both: about 2 width + 10 vector instructions per
// channel and row against 2 to 4 bytes in each direction.
#include "layer_common.hpp"

namespace {

using namespace layer;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct ConvParams {
    void* state;
    const void* x;
    void* out;
    const void* weight;
    const void* bias;
    const void* cu;
    const uint8_t* has;
    const void* slots;
    int64_t nslots, slot_stride, x_stride, out_stride, rows, dim, nseq, pad_slot_id;
    int64_t waves;          // (tile, channel block) pairs
    int32_t channel_blocks;
    int32_t tile;           // rows of a wave, at least 3 for packed prompts
    int32_t cu64, slot64, silu;
};

// Where the widened inputs of one row and the taps meet: u[0] is the oldest.
template <int VEC, int W>
__device__ __forceinline__ void taps(const float (&w)[W][VEC], const float (&bias)[VEC],
                                     const float (&u)[W - 1][VEC], const float (&now)[VEC],
                                     int silu, float (&y)[VEC]) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        float v = bias[c];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) v = fmaf(w[k][c], u[k][c], v);
        v = fmaf(w[W - 1][c], now[c], v);
        y[c] = silu ? silu_fast(v) : v;
    }
}

// The lane's taps (weight is [dim, width]: VEC * W adjacent elements) and bias: requested
// first, widened once other requests are on their way.
template <typename T, int VEC, int W>
struct Taps {
    typename Raw<T, VEC>::type raw[W], raw_bias;
    __device__ __forceinline__ void request(const ConvParams& p, int64_t c0) {
        const T* src = static_cast<const T*>(p.weight) + c0 * W;
#pragma unroll
        for (int k = 0; k < W; ++k) raw[k] = Raw<T, VEC>::load(src + k * VEC);
        // Without a bias the taps' first elements are read and not used.
        raw_bias = Raw<T, VEC>::load(p.bias ? static_cast<const T*>(p.bias) + c0 : src);
    }
    __device__ __forceinline__ void widen(const ConvParams& p, float (&w)[W][VEC],
                                          float (&bias)[VEC]) const {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            float f[VEC];
            Raw<T, VEC>::widen(raw[k], f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[(k * VEC + i) % W][(k * VEC + i) / W] = f[i];
        }
        Raw<T, VEC>::widen(raw_bias, bias);
#pragma unroll
        for (int i = 0; i < VEC; ++i) bias[i] = p.bias ? bias[i] : 0.f;
    }
};

__device__ __forceinline__ int64_t slot_of(const ConvParams& p, int64_t b) {
    const int64_t s = p.slots ? load_index(p.slots, p.slot64, b) : b;
    return s != p.pad_slot_id && s >= 0 && s < p.nslots ? s : -1;
}

// The sequences of a call as a wave sees them. Up to 63 are read at once, a lane each, and
// handed over between lanes: what a short call waits for are dependent reads.
struct Sequences {
    const ConvParams& p;
    int64_t start, slot;  // this lane's sequence: its first row, its slot or -1
    int has;
    bool few;
    __device__ __forceinline__ explicit Sequences(const ConvParams& params) : p(params) {
        const int lane = threadIdx.x & 63;
        few = p.nseq < 64;
        start = slot = has = 0;
        if (few && lane <= p.nseq) {
            start = load_index(p.cu, p.cu64, lane);
            if (lane < p.nseq) {
                slot = slot_of(p, lane);
                has = p.has && p.has[lane];
            }
        }
    }
    // The last sequence that starts at or before `row`, or -1.
    __device__ __forceinline__ int64_t at(int64_t row) const {
        if (!few) return ssu::uniform64(count_starts(p.cu, p.cu64, p.nseq, row) - 1);
        const bool in = static_cast<int>(threadIdx.x & 63) < p.nseq && start <= row;
        return __builtin_popcountll(__ballot(in)) - 1;
    }
    __device__ __forceinline__ int64_t begin(int64_t i) const {
        return few ? lane64(start, static_cast<int>(i)) : ssu::uniform64(load_index(p.cu, p.cu64, i));
    }
    __device__ __forceinline__ int64_t slot_at(int64_t i) const {
        return few ? lane64(slot, static_cast<int>(i)) : ssu::uniform64(slot_of(p, i));
    }
    __device__ __forceinline__ bool has_at(int64_t i) const {
        return few ? __builtin_amdgcn_readlane(has, static_cast<int>(i)) : p.has && p.has[i];
    }
};

// Packed prompts. A wave walks `tile` packed rows of one channel block. Where a
// sequence starts it takes the slot's history, and it stores the sequence's final
// history too, so no other wave touches that slot: a wave whose tile begins
// within the first width - 1 rows of a sequence leaves those to the wave before
// it, which goes on past its own tile for them. Inputs are requested kBatch rows
// ahead of their use, the first ones before the rows' sequences are known.
//
// Memory bounds long prompts: 17,885 rows of 10,240 channels in bf16 (733 MB) take 138 to 140 us,
// 5.3 TB/s, with tiles of 16 rows (142, 149 and 157 us with 8, 32 and 64) and outputs that
// bypass the caches (145 us without; 138 us if the inputs bypass them too). Few rows are
// latency: tiles of 4 rows then put more waves on it.
template <typename T, int VEC, int W>
__global__ __launch_bounds__(kThreads) void conv_varlen_kernel(const ConvParams p) {
    constexpr int kBatch = 8;
    typedef Raw<T, VEC> R;
    const int lane = threadIdx.x & 63;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kWaves +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (wave >= p.waves) return;
    const int64_t c0 = (wave % p.channel_blocks) * (64 * VEC) + lane * VEC;
    const int64_t r0 = wave / p.channel_blocks * p.tile;
    const int64_t r1 = r0 + p.tile < p.rows ? r0 + p.tile : p.rows;

    // Lanes past the last channel repeat the first and store nothing: the whole wave stays
    // together, since its lanes hold the sequences.
    const bool inside = c0 < p.dim;
    const int64_t c = inside ? c0 : 0;
    const T* x = static_cast<const T*>(p.x) + c;
    typename R::type raw[kBatch], before[W - 1];
    const auto request = [&](int64_t from, int64_t last) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            raw[j] = R::load(x + (from + j < last ? from + j : last - 1) * p.x_stride);
    };
    const auto request_before = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            const int64_t q = row - (W - 1) + k;
            before[k] = R::load(x + (q > 0 ? q : 0) * p.x_stride);
        }
    };
    const Sequences seqs(p);
    Taps<T, VEC, W> taps_in;
    taps_in.request(p, c);
    request_before(r0);
    request(r0, p.rows);

    // The sequence of row r0, and the rows that are this wave's.
    int64_t b = seqs.at(r0), begin = 0, end = 0, slot = -1;
    const auto enter = [&](int64_t i) {
        b = i;
        begin = seqs.begin(i);
        end = seqs.begin(i + 1);
        slot = begin >= 0 && begin <= end && end <= p.rows ? seqs.slot_at(i) : -1;
    };
    int64_t r = r0, stop = r1;
    if (b >= 0) {
        enter(b);
        if (slot >= 0 && r0 > begin && r0 < begin + W - 1) r = begin + W - 1 < end ? begin + W - 1 : end;
    }
    {
        int64_t lb = begin, le = end;
        bool ok = slot >= 0;
        if (!(b >= 0 && r1 <= le)) {
            const int64_t last = seqs.at(r1 - 1);
            ok = last >= 0;
            if (ok) {
                lb = seqs.begin(last);
                le = seqs.begin(last + 1);
                ok = lb >= 0 && lb <= le && le <= p.rows;
            }
        }
        if (ok && r1 > lb && r1 < le && r1 < lb + W - 1) stop = lb + W - 1 < le ? lb + W - 1 : le;
    }
    if (r >= stop) return;
    if (r != r0) {
        request_before(r);
        request(r, p.rows);
    }

    float w[W][VEC], bias[VEC], u[W - 1][VEC];
    taps_in.widen(p, w, bias);
    T* out = static_cast<T*>(p.out) + c;
    T* state = static_cast<T*>(p.state) + c;
    // In the middle of a sequence the rows before r are its own; else they are replaced.
#pragma unroll
    for (int k = 0; k < W - 1; ++k) R::widen(before[k], u[k]);

    const int64_t first = r;
    for (; r < stop; r += kBatch) {
        if (r != first) request(r, stop);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t row = r + j;
            if (row >= stop) break;
            while (row >= end && b + 1 < p.nseq) enter(b + 1);
            if (slot < 0 || row < begin || row >= end) continue;
            if (row == begin) {
                // The history, and the history that the sequence leaves behind.
                T* h = state + slot * p.slot_stride;
                const bool has = seqs.has_at(b);
                typename R::type old[W - 1];
#pragma unroll
                for (int k = 0; k < W - 1; ++k) {
                    typename R::type zero{};
                    old[k] = has ? R::load(h + k * p.dim) : zero;
                    R::widen(old[k], u[k]);
                }
                const int64_t len = end - begin;
#pragma unroll
                for (int k = 0; k < W - 1; ++k) {
                    const int64_t from = len - (W - 1) + k;  // position of entry k
                    typename R::type v{};
                    if (from >= 0) {
                        v = R::load(x + (begin + from) * p.x_stride);
                    } else {
#pragma unroll
                        for (int i = 0; i < W - 1; ++i)
                            if (i == from + W - 1) v = old[i];
                    }
                    if (inside) R::store(h + k * p.dim, v);
                }
            }
            float now[VEC], y[VEC];
            R::widen(raw[j], now);
            taps<VEC, W>(w, bias, u, now, p.silu, y);
            if (inside) R::store_through(out + row * p.out_stride, R::narrow(y));
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) u[k][i] = u[k + 1][i];
#pragma unroll
            for (int i = 0; i < VEC; ++i) u[W - 2][i] = now[i];
        }
    }
}

// Single tokens. A wave takes one channel block of `tile` sequences, one after the
// other, with the taps held over all of them. Memory bounds it: 512 sequences of 10,240
// channels in bf16 (84 MB) take 17 us on histories that no cache holds, 4.8 TB/s (20 us with
// histories that the caches keep: the next step finds other layers' there), with two
// sequences per wave (1 us less than one; four are no better). Small batches are
// latency and take one.
template <typename T, int VEC, int W>
__global__ __launch_bounds__(kThreads) void conv_update_kernel(const ConvParams p) {
    typedef Raw<T, VEC> R;
    const int lane = threadIdx.x & 63;
    const int64_t wave = static_cast<int64_t>(blockIdx.x) * kWaves +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (wave >= p.waves) return;
    const int64_t c0 = (wave % p.channel_blocks) * (64 * VEC) + lane * VEC;
    const int64_t b0 = wave / p.channel_blocks * p.tile;
    if (c0 >= p.dim) return;
    Taps<T, VEC, W> taps_in;
    taps_in.request(p, c0);
    float w[W][VEC], bias[VEC];
    const T* x = static_cast<const T*>(p.x) + c0;
    T* out = static_cast<T*>(p.out) + c0;
    T* state = static_cast<T*>(p.state) + c0;
    for (int64_t b = b0; b < b0 + p.tile && b < p.rows; ++b) {
        const int64_t slot = slot_of(p, b);
        if (slot < 0) continue;
        T* h = state + slot * p.slot_stride;
        typename R::type old[W - 1], fresh = R::load(x + b * p.x_stride);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) old[k] = R::load_through(h + k * p.dim);
        float u[W - 1][VEC], now[VEC], y[VEC];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) R::widen(old[k], u[k]);
        R::widen(fresh, now);
        taps_in.widen(p, w, bias);
        taps<VEC, W>(w, bias, u, now, p.silu, y);
        R::store(out + b * p.out_stride, R::narrow(y));
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) R::store_through(h + k * p.dim, old[k + 1]);
        R::store_through(h + (W - 2) * p.dim, fresh);
    }
}

int check(const ssu_conv_args* a, bool varlen) {
    using ssu::report;
    if (!a) return report(SSU_ERR_INVALID_ARGUMENT, "args must not be NULL");
    if (a->struct_size != sizeof(ssu_conv_args))
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "struct_size %u != sizeof(ssu_conv_args) %zu (header mismatch)",
                      a->struct_size, sizeof(ssu_conv_args));
    if (!is_dtype(a->io_dtype))
        return report(SSU_ERR_INVALID_ARGUMENT, "io_dtype %d is not an ssu_dtype", a->io_dtype);
    if (a->rows < 0 || a->dim < 1 || a->nslots < 1 || a->nseq < 0)
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "sizes must be positive (rows %lld, dim %lld, nslots %lld, nseq %lld)",
                      (long long)a->rows, (long long)a->dim, (long long)a->nslots,
                      (long long)a->nseq);
    if (a->width < 2 || a->width > 4)
        return report(SSU_ERR_UNSUPPORTED, "width %d is not built (2, 3 or 4)", a->width);
    if (a->x_stride < 0 || a->out_stride < a->dim)
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "x_stride must be >= 0 and out_stride at least dim");
    if (a->slot_stride < (a->width - 1) * a->dim)
        return report(SSU_ERR_INVALID_ARGUMENT, "slot_stride must be at least (width - 1) * dim");
    if (varlen && !is_index(a->cu_dtype))
        return report(SSU_ERR_INVALID_ARGUMENT, "cu_dtype %d is not an ssu_index_dtype",
                      a->cu_dtype);
    if (a->slots && !is_index(a->slot_dtype))
        return report(SSU_ERR_INVALID_ARGUMENT, "slot_dtype %d is not an ssu_index_dtype",
                      a->slot_dtype);
    if (!varlen && (a->cu_seqlens || a->has_initial))
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "cu_seqlens and has_initial belong to ssu_conv1d_varlen");
    if (!varlen && a->nseq != a->rows)
        return report(SSU_ERR_INVALID_ARGUMENT, "nseq must equal rows");
    if (a->rows == 0 || a->nseq == 0) return SSU_OK;
    const struct { const char* name; const void* p; } required[] = {
        {"conv_state", a->conv_state}, {"x", a->x}, {"out", a->out}, {"weight", a->weight}};
    for (const auto& q : required)
        if (!q.p) return report(SSU_ERR_INVALID_ARGUMENT, "%s must not be NULL", q.name);
    if (varlen && !a->cu_seqlens)
        return report(SSU_ERR_INVALID_ARGUMENT, "cu_seqlens must not be NULL");
    const int64_t esz = size_of(a->io_dtype);
    for (const void* q : {static_cast<const void*>(a->conv_state), a->x,
                          static_cast<const void*>(a->out), a->weight, a->bias})
        if (!aligned(q, esz))
            return report(SSU_ERR_INVALID_ARGUMENT, "operands must be aligned to their dtype");
    const Rows out(a->out, a->rows, a->out_stride, a->dim, esz);
    const Rows state(a->conv_state, a->nslots, a->slot_stride, (a->width - 1) * a->dim, esz);
    const struct { const char* name; Rows rows; } inputs[] = {
        {"x", Rows(a->x, a->rows, a->x_stride, a->dim, esz)},
        {"weight", Rows(a->weight, a->dim * a->width * esz)},
        {"bias", Rows(a->bias, a->dim * esz)}};
    for (const auto& in : inputs) {
        if (overlap(out, in.rows))
            return report(SSU_ERR_INVALID_ARGUMENT, "out overlaps %s", in.name);
        if (overlap(state, in.rows))
            return report(SSU_ERR_INVALID_ARGUMENT, "conv_state overlaps %s", in.name);
    }
    if (overlap(out, state))
        return report(SSU_ERR_INVALID_ARGUMENT, "out overlaps conv_state");
    return SSU_OK;
}

// Whether every row, history entry and tap block of 16 bytes is aligned.
bool wide(const ssu_conv_args* a) {
    const int64_t esz = size_of(a->io_dtype), vec = 16 / esz;
    return a->dim % vec == 0 && a->x_stride % vec == 0 && a->out_stride % vec == 0 &&
           a->slot_stride % vec == 0 && aligned(a->x, 16) && aligned(a->out, 16) &&
           aligned(a->conv_state, 16) && aligned(a->weight, 16) && aligned(a->bias, 16);
}

template <typename T, int VEC, int W, bool VARLEN>
int launch(const ssu_conv_args* a, hipStream_t stream, const char* entry) {
    ConvParams p{};
    p.state = a->conv_state;
    p.x = a->x;
    p.out = a->out;
    p.weight = a->weight;
    p.bias = a->bias;
    p.cu = a->cu_seqlens;
    p.has = a->has_initial;
    p.slots = a->slots;
    p.nslots = a->nslots;
    p.slot_stride = a->slot_stride;
    p.x_stride = a->x_stride;
    p.out_stride = a->out_stride;
    p.rows = a->rows;
    p.dim = a->dim;
    p.nseq = a->nseq;
    p.pad_slot_id = a->pad_slot_id;
    p.cu64 = a->cu_dtype == SSU_I64;
    p.slot64 = a->slot_dtype == SSU_I64;
    p.silu = a->silu != 0;
    const int64_t blocks = (a->dim + 64 * VEC - 1) / (64 * VEC);
    p.tile = VARLEN ? ((a->rows + 15) / 16 * blocks >= 2048 ? 16 : 4) : (a->rows * blocks >= 8192 ? 2 : 1);
    const int64_t tiles = (a->rows + p.tile - 1) / p.tile;
    if (blocks > INT32_MAX || tiles * blocks > static_cast<int64_t>(INT32_MAX) * kWaves)
        return ssu::report(SSU_ERR_UNSUPPORTED, "%s: too many rows for one launch", entry);
    p.channel_blocks = static_cast<int32_t>(blocks);
    p.waves = tiles * blocks;
    const dim3 grid(static_cast<unsigned>((p.waves + kWaves - 1) / kWaves));
    if constexpr (VARLEN)
        hipLaunchKernelGGL((conv_varlen_kernel<T, VEC, W>), grid, dim3(kThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((conv_update_kernel<T, VEC, W>), grid, dim3(kThreads), 0, stream, p);
    return launched(entry);
}

template <typename T, bool VARLEN>
int by_shape(const ssu_conv_args* a, hipStream_t stream, const char* entry) {
    constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    const bool w = wide(a);
    switch (a->width) {
        case 2: return w ? launch<T, kVec, 2, VARLEN>(a, stream, entry)
                         : launch<T, 1, 2, VARLEN>(a, stream, entry);
        case 3: return w ? launch<T, kVec, 3, VARLEN>(a, stream, entry)
                         : launch<T, 1, 3, VARLEN>(a, stream, entry);
        default: return w ? launch<T, kVec, 4, VARLEN>(a, stream, entry)
                          : launch<T, 1, 4, VARLEN>(a, stream, entry);
    }
}

template <bool VARLEN>
int conv(const ssu_conv_args* a, void* stream, const char* entry) {
    if (int rc = check(a, VARLEN)) return rc;
    if (a->rows == 0 || a->nseq == 0) return ssu::report_ok();
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (a->io_dtype) {
        case SSU_F32: return by_shape<float, VARLEN>(a, s, entry);
        case SSU_F16: return by_shape<_Float16, VARLEN>(a, s, entry);
        default: return by_shape<__bf16, VARLEN>(a, s, entry);
    }
}

}  // namespace

extern "C" {

int ssu_conv1d_varlen(const ssu_conv_args* a, void* stream) {
    return conv<true>(a, stream, "ssu_conv1d_varlen");
}

int ssu_conv1d_update(const ssu_conv_args* a, void* stream) {
    return conv<false>(a, stream, "ssu_conv1d_update");
}

}  // extern "C"
