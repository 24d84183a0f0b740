// layer_common.hpp -- what the kernels and front ends of the layer operators
// (include/layer.h) share: element access by storage type, the search for a
// packed row's sequence, and host-side checks of argument structs.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.h"
#include "ssu_kernel.hpp"
#include "ssu_launch.h"

namespace layer {

using ssu::Bits;
using ssu::Pack;
using ssu::Words;
using ssu::group_sum;
using ssu::lds_barrier;
using ssu::load_index;
using ssu::widen_io;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// VEC consecutive elements of storage type T as 32-bit words (one 16-bit value in
// a half word when VEC is 1), moved by one vector-memory instruction.
template <typename T, int VEC>
struct Raw {
    static constexpr int kWords = VEC * static_cast<int>(sizeof(T)) / 4;
    typedef typename ssu::Words<kWords>::type type;
    static __device__ __forceinline__ type load(const T* p) {
        return *reinterpret_cast<const type*>(p);
    }
    static __device__ __forceinline__ void store(T* p, type v) { *reinterpret_cast<type*>(p) = v; }
    // Past the caches: for what is not read again before much else is.
    static __device__ __forceinline__ type load_through(const T* p) {
        return __builtin_nontemporal_load(reinterpret_cast<const type*>(p));
    }
    static __device__ __forceinline__ void store_through(T* p, type v) {
        __builtin_nontemporal_store(v, reinterpret_cast<type*>(p));
    }
    static __device__ __forceinline__ void widen(type v, float (&f)[VEC]) {
        constexpr int per = ssu::Pack<T>::kPerWord;
#pragma unroll
        for (int i = 0; i < kWords; ++i) ssu::Pack<T>::widen(word(v, i), &f[i * per]);
    }
    static __device__ __forceinline__ type narrow(const float (&f)[VEC]) {
        constexpr int per = ssu::Pack<T>::kPerWord;
        type v;
        if constexpr (kWords == 1) {
            v[0] = ssu::Pack<T>::narrow(&f[0]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) v[i] = ssu::Pack<T>::narrow(&f[i * per]);
        }
        return v;
    }
    static __device__ __forceinline__ unsigned word(type v, int i) { return v[i]; }
};

template <typename T>
struct Raw<T, 1> {
    typedef typename ssu::Bits<T>::type type;
    static __device__ __forceinline__ type load(const T* p) {
        return *reinterpret_cast<const type*>(p);
    }
    static __device__ __forceinline__ void store(T* p, type v) { *reinterpret_cast<type*>(p) = v; }
    // Past the caches: for what is not read again before much else is.
    static __device__ __forceinline__ type load_through(const T* p) {
        return __builtin_nontemporal_load(reinterpret_cast<const type*>(p));
    }
    static __device__ __forceinline__ void store_through(T* p, type v) {
        __builtin_nontemporal_store(v, reinterpret_cast<type*>(p));
    }
    static __device__ __forceinline__ void widen(type v, float (&f)[1]) {
        f[0] = ssu::widen_io<T>(v);
    }
    static __device__ __forceinline__ type narrow(const float (&f)[1]) {
        return __builtin_bit_cast(type, static_cast<T>(f[0]));
    }
};

// v * sigmoid(v) with the hardware's exp2 and reciprocal (each within about one
// unit in the last place). The exponent's argument is rounded, which grows with it: an fp32
// result is off by up to (6 + 3 |v|) 2^-24 relative, far below one rounding of a 16-bit
// result until sigmoid is 2^-126. Minus infinity gives NaN as the formula does.
__device__ __forceinline__ float silu_fast(float v) {
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * v));
}

// The number of entries i < n of the non-decreasing cu with cu[i] <= row, found by
// the whole wave: every step probes 64 entries and keeps the interval between two
// of them, so it ends for any content of cu.
__device__ __forceinline__ int64_t count_starts(const void* cu, int is64, int64_t n, int64_t row) {
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t step = (hi - lo + 63) / 64;
        const int64_t i = lo + lane * step;
        const bool in = i < hi && load_index(cu, is64, i) <= row;
        const int c = __builtin_popcountll(__ballot(in));
        if (step == 1) return lo + c;
        if (c == 0) return lo;
        hi = lo + c * step < hi ? lo + c * step : hi;
        lo += (c - 1) * step + 1;
    }
    return lo;
}

// The 64-bit value of lane i, the same for the whole wave.
__device__ __forceinline__ int64_t lane64(int64_t v, int i) {
    const unsigned lo = __builtin_amdgcn_readlane(static_cast<unsigned>(v), i);
    const unsigned hi = __builtin_amdgcn_readlane(static_cast<unsigned>(v >> 32), i);
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// ------------------------------------------------------------------ host checks

inline bool is_dtype(int32_t d) { return d == SSU_F32 || d == SSU_F16 || d == SSU_BF16; }
inline bool is_index(int32_t d) { return d == SSU_I32 || d == SSU_I64; }
inline int64_t size_of(int32_t d) { return d == SSU_F32 ? 4 : 2; }
inline bool aligned(const void* p, int64_t a) {
    return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(a) == 0;
}

// An operand's bytes: `n` rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t n, stride, width;
    Rows(const void* base, int64_t rows, int64_t stride_elements, int64_t elements, int64_t esz)
        : p(base), n(rows), stride(stride_elements * esz), width(elements * esz) {}
    Rows(const void* base, int64_t bytes) : p(base), n(1), stride(0), width(bytes) {}
    int64_t span() const { return n > 0 ? (n - 1) * stride + width : 0; }
};

// Whether two operands share a byte; for those of unequal strides whether their spans do.
inline bool overlap(const Rows& a, const Rows& b) {
    if (!a.p || !b.p || a.span() <= 0 || b.span() <= 0) return false;
    const auto a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    if (a0 >= b0 + static_cast<uintptr_t>(b.span()) || b0 >= a0 + static_cast<uintptr_t>(a.span()))
        return false;
    // Rows of one stride (a single row has any): b's columns may lie beside a's.
    const int64_t stride = a.n > 1 ? a.stride : b.stride;
    if (stride <= 0 || (b.n > 1 && b.stride != stride)) return true;
    const auto s = static_cast<uintptr_t>(stride);
    const int64_t at = static_cast<int64_t>(b0 >= a0 ? (b0 - a0) % s : (s - (a0 - b0) % s) % s);
    return at < a.width || at + b.width > stride;
}

inline int launched(const char* entry) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return ssu::report(SSU_ERR_LAUNCH, "%s: launch failed: %s", entry, hipGetErrorString(e));
    return ssu::report_ok();
}

}  // namespace layer
