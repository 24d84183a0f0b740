// layer_cache.hip -- slots of state caches: allocation, freeing, copying and
// compaction (semantics in include/layer.h).
//
// The counters are integers and small (one per slot of a cache), so one workgroup
// walks them with a running prefix count; no atomics order anything, and every
// result is the same from run to run. The copies are the work: 16 bytes per lane,
// four in flight, bounded by memory. A source slot that several neighbouring pairs
// name (a prompt answered several ways) is read once and written to each.
#include "layer_common.hpp"

namespace {

using namespace layer;

// ---------------------------------------------------------------- the counters

constexpr int kScan = 1024;
constexpr int kScanWaves = kScan / 64;

// For the workgroup's kScan flags: the number of set flags before this thread's,
// and the total. `shared` holds kScanWaves + 1 entries.
__device__ __forceinline__ int prefix(bool flag, int* shared, int* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const unsigned long long m = __ballot(flag);
    __syncthreads();  // the previous use of shared has ended
    if (lane == 0) shared[wave] = __builtin_popcountll(m);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kScanWaves; ++w) {
        const int c = shared[w];
        before += w < wave ? c : 0;
        all += c;
    }
    *total = all;
    return before + __builtin_popcountll(m & ((1ull << lane) - 1));
}

__global__ __launch_bounds__(kScan) void alloc_kernel(int32_t* refcount, int64_t nslots,
                                                      int32_t* ids, int64_t n) {
    __shared__ int shared[kScanWaves];
    int64_t found = 0;
    for (int64_t base = 0; base < nslots && found < n; base += kScan) {
        const int64_t i = base + threadIdx.x;
        const bool free = i < nslots && refcount[i] <= 0;
        int total;
        const int64_t at = found + prefix(free, shared, &total);
        if (free && at < n) {
            ids[at] = static_cast<int32_t>(i);
            refcount[i] = 1;
        }
        found += total;
    }
    for (int64_t i = found + threadIdx.x; i < n; i += kScan) ids[i] = -1;
}

// A slot may be named more than once, so counts change atomically; they are
// integers, and the result does not depend on the order: a free slot stays free,
// and a count never passes below zero on the way down.
__global__ void adjust_kernel(int32_t* refcount, int64_t nslots, const void* slots, int is64,
                              int64_t n, int32_t delta) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t s = load_index(slots, is64, i);
    if (s < 0 || s >= nslots) return;
    int32_t old = __hip_atomic_load(&refcount[s], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    while (old > 0 && !__hip_atomic_compare_exchange_strong(&refcount[s], &old, old + delta,
                                                            __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                                            __HIP_MEMORY_SCOPE_AGENT)) {
    }
}

// plan[0] = number of moves m; plan[1 + k] = the slot that move k leaves; plan[1 +
// half + k] = the slot it fills, half = nslots / 2 >= m.
__global__ __launch_bounds__(kScan) void plan_kernel(int32_t* refcount, int64_t nslots,
                                                     int32_t* remap, int32_t* plan) {
    __shared__ int shared[kScanWaves];
    int64_t live = 0;
    for (int64_t base = 0; base < nslots; base += kScan) {
        const int64_t i = base + threadIdx.x;
        int total;
        prefix(i < nslots && refcount[i] > 0, shared, &total);
        live += total;
    }
    int32_t* leave = plan + 1;
    int32_t* fill = plan + 1 + nslots / 2;
    int64_t holes = 0, movers = 0;
    for (int64_t base = 0; base < nslots; base += kScan) {
        const int64_t i = base + threadIdx.x;
        const bool used = i < nslots && refcount[i] > 0;
        const bool hole = i < live && !used, mover = i >= live && used;
        int total;
        const int64_t h = holes + prefix(hole, shared, &total);
        holes += total;
        const int64_t m = movers + prefix(mover, shared, &total);
        movers += total;
        if (hole) fill[h] = static_cast<int32_t>(i);
        if (mover) leave[m] = static_cast<int32_t>(i);
        if (i < nslots && !mover) remap[i] = used ? static_cast<int32_t>(i) : -1;
    }
    // As many slots in use lie above `live` as free ones below it.
    if (threadIdx.x == 0) plan[0] = static_cast<int32_t>(movers);
    __threadfence_block();
    __syncthreads();
    for (int64_t k = threadIdx.x; k < movers; k += kScan) {
        const int32_t from = leave[k], to = fill[k];
        remap[from] = to;
        refcount[to] = refcount[from];
        refcount[from] = 0;
    }
}

// ---------------------------------------------------------------------- copies

constexpr int kThreads = 256;
constexpr int kDepth = 4;                              // loads in flight per lane and pair
constexpr int kPairs = 4;                              // neighbouring pairs of a workgroup, where there are many
constexpr int64_t kTile = kThreads * kDepth * 16;      // bytes of a slot per workgroup
constexpr int64_t kMostItems = INT32_MAX / 2;          // (tile, group) pairs of one launch
constexpr int64_t kFewItems = 1024;                    // (tile, pair) pairs
constexpr int kMaxCaches = 32;                         // caches of one launch

struct Block {
    char* base;
    int64_t slot_bytes, stride;
};

struct CopyParams {
    const void* src;
    const void* dst;
    const int32_t* plan;  // compaction: moves in plan_kernel's layout, else NULL
    int64_t first, n;     // pairs of this launch (of a plan's: at most)
    int64_t nslots, half;
    int32_t tiles;        // of a slot in all caches
    int32_t src64, dst64, ncaches;
    uint32_t wide;        // bit i: cache[i] moves 16 bytes at a time
    int32_t first_tile[kMaxCaches];
    Block cache[kMaxCaches];
};

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// One tile of one slot (bytes [at, at + kTile) of it, cut at its end): the four
// 16-byte pieces of a lane, or where a cache's slots are not 16-byte aligned its
// bytes one by one.
template <int PAIRS>
__device__ __forceinline__ void copy_tile(const Block& c, int64_t at, const int (&from)[PAIRS],
                                          const int (&to)[PAIRS], bool wide) {
    if (wide) {
        u32x4 v[PAIRS][kDepth];
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            if (from[k] < 0) continue;
            if (k > 0 && from[k] == from[k - 1]) {
#pragma unroll
                for (int j = 0; j < kDepth; ++j) v[k][j] = v[k - 1][j];
                continue;
            }
#pragma unroll
            for (int j = 0; j < kDepth; ++j) {
                const int64_t o = at + (j * kThreads + threadIdx.x) * 16;
                if (o < c.slot_bytes)
                    v[k][j] = __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4*>(c.base + from[k] * c.stride + o));
            }
        }
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            if (from[k] < 0) continue;
#pragma unroll
            for (int j = 0; j < kDepth; ++j) {
                const int64_t o = at + (j * kThreads + threadIdx.x) * 16;
                if (o < c.slot_bytes)
                    __builtin_nontemporal_store(
                        v[k][j], reinterpret_cast<u32x4*>(c.base + to[k] * c.stride + o));
            }
        }
    } else {
        const int64_t end = at + kTile < c.slot_bytes ? at + kTile : c.slot_bytes;
        for (int k = 0; k < PAIRS; ++k) {
            if (from[k] < 0) continue;
            for (int64_t o = at + threadIdx.x; o < end; o += kThreads)
                c.base[to[k] * c.stride + o] = c.base[from[k] * c.stride + o];
        }
    }
}

// Items are (group of pairs, tile), tiles of a group adjacent, and every XCD walks a
// contiguous range of them: 16 parents forked four ways over 16 caches (2.7 GB) take 523 us
// so, 545 us in the hardware's order, 811 us with one pair at a time. Plain loads and
// stores take 510 us there and 145 instead of 136 us on 36 moves of 10.6 MB; kept are those
// that leave the caches to others. (A copy streams at 5.4 TB/s, a fill at 5.6.)
template <int PAIRS>
__global__ __launch_bounds__(kThreads) void copy_kernel(const CopyParams p) {
    const int lane = threadIdx.x & 63;
    int64_t n = p.n;
    if (p.plan) n = p.plan[0] - p.first < n ? p.plan[0] - p.first : n;
    const int first_tile = lane < p.ncaches ? p.first_tile[lane] : 0x7fffffff;
    const int items = static_cast<int>((n + PAIRS - 1) / PAIRS) * p.tiles;
    for (int k = blockIdx.x; k < items; k += gridDim.x) {
        const int item = static_cast<int>(ssu::xcd_tile(k, items));
        const int group = item / p.tiles, tile = item % p.tiles;
        const int ci = __builtin_popcountll(__ballot(first_tile <= tile)) - 1;
        const Block c = p.cache[ci];
        const int64_t in_slot = static_cast<int64_t>(tile - __builtin_amdgcn_readlane(first_tile, ci)) * kTile;
        // Lane k < PAIRS reads pair k's ids: one wait for all of them.
        const int64_t mine = static_cast<int64_t>(group) * PAIRS + lane, at = p.first + mine;
        int from_lane = -1, to_lane = -1;
        if (lane < PAIRS && mine < n) {
            const int64_t s = p.plan ? p.plan[1 + at] : load_index(p.src, p.src64, at);
            const int64_t d = p.plan ? p.plan[1 + p.half + at] : load_index(p.dst, p.dst64, at);
            if (s >= 0 && s < p.nslots && d >= 0 && d < p.nslots && s != d) {
                from_lane = static_cast<int>(s);
                to_lane = static_cast<int>(d);
            }
        }
        int from[PAIRS], to[PAIRS];
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
            from[k] = __builtin_amdgcn_readlane(from_lane, k);
            to[k] = __builtin_amdgcn_readlane(to_lane, k);
        }
        copy_tile(c, in_slot, from, to, p.wide >> ci & 1);
    }
}

int check(const ssu_cache_args* a) {
    using ssu::report;
    if (!a) return report(SSU_ERR_INVALID_ARGUMENT, "args must not be NULL");
    if (a->struct_size != sizeof(ssu_cache_args))
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "struct_size %u != sizeof(ssu_cache_args) %zu (header mismatch)",
                      a->struct_size, sizeof(ssu_cache_args));
    if (a->nslots < 0 || a->nslots > INT32_MAX)
        return report(SSU_ERR_INVALID_ARGUMENT, "nslots must be in [0, 2^31), got %lld",
                      (long long)a->nslots);
    if (a->n < 0 || a->n > INT32_MAX)
        return report(SSU_ERR_INVALID_ARGUMENT, "n must be in [0, 2^31), got %lld",
                      (long long)a->n);
    return SSU_OK;
}

int check_counts(const ssu_cache_args* a) {
    if (a->nslots > 0 && !a->refcount)
        return ssu::report(SSU_ERR_INVALID_ARGUMENT, "refcount must not be NULL");
    if (!aligned(a->refcount, 4))
        return ssu::report(SSU_ERR_INVALID_ARGUMENT, "refcount must be aligned to its dtype");
    return SSU_OK;
}

int check_ids(const char* name, const void* p, int32_t dtype) {
    if (!is_index(dtype))
        return ssu::report(SSU_ERR_INVALID_ARGUMENT, "%s_dtype %d is not an ssu_index_dtype", name,
                           dtype);
    if (!p) return ssu::report(SSU_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
    if (!aligned(p, dtype == SSU_I64 ? 8 : 4))
        return ssu::report(SSU_ERR_INVALID_ARGUMENT, "%s must be aligned to its dtype", name);
    return SSU_OK;
}

int check_caches(const ssu_cache_args* a) {
    using ssu::report;
    if (a->ncaches < 0) return report(SSU_ERR_INVALID_ARGUMENT, "ncaches must be >= 0");
    if (a->ncaches > 0 && !a->caches)
        return report(SSU_ERR_INVALID_ARGUMENT, "caches must not be NULL");
    for (int64_t i = 0; i < a->ncaches; ++i) {
        const ssu_cache_block& c = a->caches[i];
        if (c.slot_bytes < 0 || c.stride_bytes < c.slot_bytes)
            return report(SSU_ERR_INVALID_ARGUMENT,
                          "cache %lld: stride_bytes must be at least slot_bytes >= 0",
                          (long long)i);
        if (c.slot_bytes > 0 && a->nslots > 0 && !c.base)
            return report(SSU_ERR_INVALID_ARGUMENT, "cache %lld: base must not be NULL",
                          (long long)i);
    }
    return SSU_OK;
}

// Copies of n pairs (or of a plan's, at most n) in every cache, kMaxCaches at a time.
int copy(const ssu_cache_args* a, const int32_t* plan, const void* src, int src64, const void* dst,
         int dst64, int64_t n, hipStream_t stream, const char* entry) {
    for (int64_t done = 0; done < a->ncaches;) {
        CopyParams p{};
        p.src = src;
        p.dst = dst;
        p.src64 = src64;
        p.dst64 = dst64;
        p.plan = plan;
        p.nslots = a->nslots;
        p.half = a->nslots / 2;
        while (done < a->ncaches && p.ncaches < kMaxCaches) {
            const ssu_cache_block& c = a->caches[done];
            const int64_t tiles = (c.slot_bytes + kTile - 1) / kTile;
            if (tiles > kMostItems - p.tiles) {
                if (p.ncaches == 0)
                    return ssu::report(SSU_ERR_UNSUPPORTED, "%s: a slot of %lld bytes is too large",
                                       entry, (long long)c.slot_bytes);
                break;
            }
            ++done;
            if (tiles == 0) continue;
            p.cache[p.ncaches] = {static_cast<char*>(c.base), c.slot_bytes, c.stride_bytes};
            p.first_tile[p.ncaches] = p.tiles;
            p.tiles += static_cast<int32_t>(tiles);
            if (aligned(c.base, 16) && c.slot_bytes % 16 == 0 && c.stride_bytes % 16 == 0)
                p.wide |= 1u << p.ncaches;
            ++p.ncaches;
        }
        if (p.ncaches == 0) continue;
        // Few copies are latency: a pair per workgroup then (one request forked four ways over
        // four small caches: 4.4 us against 5.9), else kPairs (527 us against 811).
        const bool few = n * p.tiles <= kFewItems;
        const int64_t pairs = few ? 1 : kPairs;
        // The kernel counts its items in 32 bits.
        const int64_t most = kMostItems / p.tiles * pairs;
        for (p.first = 0; p.first < n; p.first += most) {
            p.n = n - p.first < most ? n - p.first : most;
            const int64_t items = (p.n + pairs - 1) / pairs * p.tiles;
            // One item per workgroup, but for compactions, whose moves are known on the
            // device only and may be few: there the grid is bounded.
            const dim3 grid(static_cast<unsigned>(plan && items > 65536 ? 65536 : items));
            if (few)
                hipLaunchKernelGGL(copy_kernel<1>, grid, dim3(kThreads), 0, stream, p);
            else
                hipLaunchKernelGGL(copy_kernel<kPairs>, grid, dim3(kThreads), 0, stream, p);
            if (int rc = launched(entry)) return rc;
        }
    }
    return ssu::report_ok();
}

}  // namespace

extern "C" {

int ssu_cache_alloc(const ssu_cache_args* a, void* stream) {
    if (int rc = check(a)) return rc;
    if (int rc = check_counts(a)) return rc;
    if (a->n == 0) return ssu::report_ok();
    if (!a->ids) return ssu::report(SSU_ERR_INVALID_ARGUMENT, "ids must not be NULL");
    hipLaunchKernelGGL(alloc_kernel, dim3(1), dim3(kScan), 0, static_cast<hipStream_t>(stream),
                       a->refcount, a->nslots, a->ids, a->n);
    return launched("ssu_cache_alloc");
}

int ssu_cache_adjust(const ssu_cache_args* a, void* stream) {
    if (int rc = check(a)) return rc;
    if (int rc = check_counts(a)) return rc;
    if (a->delta != 1 && a->delta != -1)
        return ssu::report(SSU_ERR_INVALID_ARGUMENT, "delta must be 1 or -1, got %d", a->delta);
    if (a->n == 0) return ssu::report_ok();
    if (int rc = check_ids("src", a->src, a->src_dtype)) return rc;
    const unsigned grid = static_cast<unsigned>((a->n + 255) / 256);
    hipLaunchKernelGGL(adjust_kernel, dim3(grid), dim3(256), 0, static_cast<hipStream_t>(stream),
                       a->refcount, a->nslots, a->src, a->src_dtype == SSU_I64, a->n, a->delta);
    return launched("ssu_cache_adjust");
}

int ssu_cache_copy(const ssu_cache_args* a, void* stream) {
    if (int rc = check(a)) return rc;
    if (int rc = check_caches(a)) return rc;
    if (a->n == 0 || a->nslots == 0) return ssu::report_ok();
    if (int rc = check_ids("src", a->src, a->src_dtype)) return rc;
    if (int rc = check_ids("dst", a->dst, a->dst_dtype)) return rc;
    return copy(a, nullptr, a->src, a->src_dtype == SSU_I64, a->dst, a->dst_dtype == SSU_I64, a->n,
                static_cast<hipStream_t>(stream), "ssu_cache_copy");
}

int ssu_cache_compact(const ssu_cache_args* a, void* stream) {
    if (int rc = check(a)) return rc;
    if (int rc = check_counts(a)) return rc;
    if (int rc = check_caches(a)) return rc;
    if (a->nslots == 0) return ssu::report_ok();
    if (!a->remap || !a->plan)
        return ssu::report(SSU_ERR_INVALID_ARGUMENT, "remap and plan must not be NULL");
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kScan), 0, s, a->refcount, a->nslots, a->remap,
                       a->plan);
    if (int rc = launched("ssu_cache_compact")) return rc;
    if (a->nslots < 2) return ssu::report_ok();
    return copy(a, a->plan, nullptr, 0, nullptr, 0, a->nslots / 2, s, "ssu_cache_compact");
}

}  // extern "C"
