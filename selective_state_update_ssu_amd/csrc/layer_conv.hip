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
    int32_t tile;           // rows of a wave
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

// The lane's taps (weight is [dim, width]: VEC * W adjacent elements) and bias.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvParams& p, int64_t c0, float (&w)[W][VEC],
                                          float (&bias)[VEC]) {
    const T* src = static_cast<const T*>(p.weight) + c0 * W;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float f[VEC];
        Raw<T, VEC>::widen(Raw<T, VEC>::load(src + k * VEC), f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[(k * VEC + i) % W][(k * VEC + i) / W] = f[i];
    }
    if (p.bias) {
        Raw<T, VEC>::widen(Raw<T, VEC>::load(static_cast<const T*>(p.bias) + c0), bias);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) bias[i] = 0.f;
    }
}

__device__ __forceinline__ int64_t slot_of(const ConvParams& p, int64_t b) {
    const int64_t s = p.slots ? load_index(p.slots, p.slot64, b) : b;
    return s != p.pad_slot_id && s >= 0 && s < p.nslots ? s : -1;
}

// Packed prompts. A wave walks `tile` packed rows of one channel block. Where a
// sequence starts it takes the slot's history, and it stores the sequence's final
// history too, so no other wave touches that slot: a wave whose tile begins
// within the first width - 1 rows of a sequence leaves those to the wave before
// it, which goes on past its own tile for them. Inputs are requested kBatch rows
// ahead of their use.
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

    // The sequence of row r0, and the rows that are this wave's.
    int64_t b = count_starts(p.cu, p.cu64, p.nseq, r0) - 1;
    b = ssu::uniform64(b);
    int64_t begin = 0, end = 0, slot = -1;
    const auto enter = [&](int64_t i) {
        b = i;
        begin = load_index(p.cu, p.cu64, i);
        end = load_index(p.cu, p.cu64, i + 1);
        slot = begin >= 0 && begin <= end && end <= p.rows ? slot_of(p, i) : -1;
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
            const int64_t last = ssu::uniform64(count_starts(p.cu, p.cu64, p.nseq, r1 - 1) - 1);
            if (last >= 0) {
                lb = load_index(p.cu, p.cu64, last);
                le = load_index(p.cu, p.cu64, last + 1);
                ok = lb >= 0 && lb <= le && le <= p.rows;
            } else {
                ok = false;
            }
        }
        if (ok && r1 > lb && r1 < le && r1 < lb + W - 1) stop = lb + W - 1 < le ? lb + W - 1 : le;
    }
    if (c0 >= p.dim || r >= stop) return;

    float w[W][VEC], bias[VEC], u[W - 1][VEC];
    load_taps<T, VEC, W>(p, c0, w, bias);
    const T* x = static_cast<const T*>(p.x) + c0;
    T* out = static_cast<T*>(p.out) + c0;
    T* state = static_cast<T*>(p.state) + c0;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        // In the middle of a sequence the rows before r are all its own.
        const int64_t q = r - (W - 1) + k;
        if (b >= 0 && slot >= 0 && r < end && q >= begin) {
            R::widen(R::load(x + q * p.x_stride), u[k]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) u[k][i] = 0.f;
        }
    }

    for (; r < stop; r += kBatch) {
        typename R::type raw[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t row = r + j < stop ? r + j : stop - 1;
            raw[j] = R::load(x + row * p.x_stride);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t row = r + j;
            if (row >= stop) break;
            while (row >= end && b + 1 < p.nseq) enter(b + 1);
            if (slot < 0 || row < begin || row >= end) continue;
            if (row == begin) {
                // The history, and the history that the sequence leaves behind.
                T* h = state + slot * p.slot_stride;
                const bool has = p.has && p.has[b];
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
                    R::store(h + k * p.dim, v);
                }
            }
            float now[VEC], y[VEC];
            R::widen(raw[j], now);
            taps<VEC, W>(w, bias, u, now, p.silu, y);
            R::store_through(out + row * p.out_stride, R::narrow(y));
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
// other, with the taps held over all of them.
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
    float w[W][VEC], bias[VEC];
    load_taps<T, VEC, W>(p, c0, w, bias);
    const T* x = static_cast<const T*>(p.x) + c0;
    T* out = static_cast<T*>(p.out) + c0;
    T* state = static_cast<T*>(p.state) + c0;
    for (int64_t b = b0; b < b0 + p.tile && b < p.rows; ++b) {
        const int64_t slot = slot_of(p, b);
        if (slot < 0) continue;
        T* h = state + slot * p.slot_stride;
        typename R::type old[W - 1], fresh = R::load(x + b * p.x_stride);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) old[k] = R::load(h + k * p.dim);
        float u[W - 1][VEC], now[VEC], y[VEC];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) R::widen(old[k], u[k]);
        R::widen(fresh, now);
        taps<VEC, W>(w, bias, u, now, p.silu, y);
        R::store(out + b * p.out_stride, R::narrow(y));
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) R::store(h + k * p.dim, old[k + 1]);
        R::store(h + (W - 2) * p.dim, fresh);
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
    const int64_t xb = span(a->rows, a->x_stride, a->dim, esz);
    const int64_t ob = span(a->rows, a->out_stride, a->dim, esz);
    const int64_t sb = span(a->nslots, a->slot_stride, (a->width - 1) * a->dim, esz);
    const struct { const char* name; const void* p; int64_t bytes; } inputs[] = {
        {"x", a->x, xb}, {"weight", a->weight, a->dim * a->width * esz},
        {"bias", a->bias, a->dim * esz}};
    for (const auto& in : inputs) {
        if (overlap(a->out, ob, in.p, in.bytes))
            return report(SSU_ERR_INVALID_ARGUMENT, "out overlaps %s", in.name);
        if (overlap(a->conv_state, sb, in.p, in.bytes))
            return report(SSU_ERR_INVALID_ARGUMENT, "conv_state overlaps %s", in.name);
    }
    if (overlap(a->out, ob, a->conv_state, sb))
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
    p.tile = VARLEN ? 16 : 1;
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
