// batch_plan.hip -- tables of a packed batch from its lengths (semantics in include/batch.h).
//
// One launch. Every workgroup sums the lengths (2,048 at a time, a running sum of rows and of
// chunks) and fills one stretch of a table: of the rows, or of the chunks; each entry is
// found by bisection among the sums in LDS. The first workgroup writes what there is one of per
// request. Summing again in every workgroup costs less than a second launch, which would
// have to wait for the sums: the call is latency. 5 requests: 5.9 us; 2,000 with 130,001
// rows, chunks and slots: 7.7 us (10.7 with one request per thread, 8.3 with four, which costs the
// few requests 0.4; 14.6 with four entries of a table per thread and 64-bit divisions).
#include "batch.h"
#include "layer_common.hpp"

namespace {

using namespace layer;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kStretch = kThreads;  // entries of a table per workgroup
constexpr int kEach = 2, kHeld = kEach * kThreads;  // requests of a thread, of a pass

struct PlanParams {
    const void* lengths;
    const void* context;
    const void* table;
    int32_t *cu, *row_seq, *row_pos, *cu_chunk, *seq_idx, *last;
    int64_t* row_slots;
    int64_t nseq, rows, chunk, nchunks, table_stride, table_width, block_size;
    int32_t row_blocks, length64, context64, table64;
};

// x / y for x >= 0, y > 0: a division of 64 bits takes five times as long as one of 32.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}

// Running sums of a pair over the workgroup, exclusive, and the totals.
__device__ __forceinline__ void prefix2(int64_t (&v)[2], int64_t (&total)[2], int64_t (*waves)[2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    int64_t run[2] = {v[0], v[1]};
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t below = __shfl_up(run[k], d);
            if (lane >= d) run[k] += below;
        }
    __syncthreads();  // the previous use of waves has ended
    if (lane == 63) {
        waves[wave][0] = run[0];
        waves[wave][1] = run[1];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        int64_t before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int64_t x = waves[w][k];
            before += w < wave ? x : 0;
            all += x;
        }
        v[k] = before + run[k] - v[k];
        total[k] = all;
    }
}

__global__ __launch_bounds__(kThreads) void plan_kernel(const PlanParams p) {
    __shared__ int64_t waves[kWaves][2];
    __shared__ int64_t starts[2][kHeld + 1];  // of the requests at hand: first row, first chunk
    const bool chunks = static_cast<int>(blockIdx.x) >= p.row_blocks;
    const int64_t stretch = chunks ? blockIdx.x - p.row_blocks : blockIdx.x;
    const int64_t lo = stretch * kStretch;
    const int64_t most = chunks ? p.nchunks + 1 : p.rows;
    const int64_t hi = lo + kStretch < most ? lo + kStretch : most;
    int64_t base[2] = {0, 0};
    for (int64_t b0 = 0; b0 < p.nseq; b0 += kHeld) {
        const int own = threadIdx.x * kEach;
        int64_t length[kEach] = {}, cut[kEach] = {}, at[2] = {0, 0}, total[2];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (b0 + own + k >= p.nseq) continue;
            length[k] = load_index(p.lengths, p.length64, b0 + own + k);
            if (length[k] < 0) length[k] = 0;
            if (p.chunk > 0) cut[k] = length[k] < 1 ? 1 : 1 + quotient(length[k] - 1, p.chunk);
            at[0] += length[k];
            at[1] += cut[k];
        }
        prefix2(at, total, waves);
        at[0] += base[0];
        at[1] += base[1];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int64_t b = b0 + own + k;
            starts[0][own + k] = at[0];
            starts[1][own + k] = at[1];
            if (blockIdx.x == 0 && b < p.nseq) {
                if (p.cu) p.cu[b] = static_cast<int32_t>(at[0]);
                if (p.last) {
                    const int64_t c = at[1] + cut[k] - 1;
                    p.last[b] = c < p.nchunks ? static_cast<int32_t>(c) : -1;
                }
            }
            at[0] += length[k];
            at[1] += cut[k];
        }
        if (threadIdx.x == 0) {
            starts[0][kHeld] = base[0] + total[0];
            starts[1][kHeld] = base[1] + total[1];
        }
        __syncthreads();
        // Entries of these requests in the stretch.
        const int64_t* s = starts[chunks ? 1 : 0];
        const int64_t from = s[0] > lo ? s[0] : lo;
        const int64_t end = s[kHeld] < hi ? s[kHeld] : hi;
        const int held = static_cast<int>(p.nseq - b0 < kHeld ? p.nseq - b0 : kHeld);
        for (int64_t i = from + threadIdx.x; i < end; i += kThreads) {
            int x = 0, y = held;  // s[x] <= i < s[y]
            while (y - x > 1) {
                const int m = (x + y) / 2;
                if (s[m] <= i)
                    x = m;
                else
                    y = m;
            }
            const int64_t seq = b0 + x, place = i - s[x];
            if (chunks) {
                const int64_t row = starts[0][x] + place * p.chunk;
                if (p.cu_chunk) p.cu_chunk[i] = static_cast<int32_t>(row);
                if (p.seq_idx && i < p.nchunks) p.seq_idx[i] = static_cast<int32_t>(seq);
            } else {
                const int64_t pos =
                    place + (p.context ? load_index(p.context, p.context64, seq) : 0);
                if (p.row_seq) p.row_seq[i] = static_cast<int32_t>(seq);
                if (p.row_pos) p.row_pos[i] = static_cast<int32_t>(pos);
                if (p.row_slots) {
                    const int64_t column = pos < 0 ? p.table_width : quotient(pos, p.block_size);
                    int64_t block = -1;
                    if (column < p.table_width)
                        block = load_index(p.table, p.table64, seq * p.table_stride + column);
                    p.row_slots[i] = block < 0 ? -1 : (block - column) * p.block_size + pos;
                }
            }
        }
        base[0] += total[0];
        base[1] += total[1];
    }
    // Behind the last request.
    const int64_t used = chunks ? base[1] : base[0];
    for (int64_t i = (used > lo ? used : lo) + threadIdx.x; i < hi; i += kThreads) {
        if (chunks) {
            if (p.cu_chunk) p.cu_chunk[i] = static_cast<int32_t>(base[0]);
            if (p.seq_idx && i < p.nchunks) p.seq_idx[i] = -1;
        } else {
            if (p.row_seq) p.row_seq[i] = -1;
            if (p.row_pos) p.row_pos[i] = -1;
            if (p.row_slots) p.row_slots[i] = -1;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.cu) p.cu[p.nseq] = static_cast<int32_t>(base[0]);
}

int check(const ssu_plan_args* a) {
    using ssu::report;
    constexpr int kBad = SSU_ERR_INVALID_ARGUMENT;
    if (!a) return report(kBad, "args must not be NULL");
    if (a->struct_size != sizeof(ssu_plan_args))
        return report(kBad, "struct_size %u != sizeof(ssu_plan_args) %zu (header mismatch)",
                      a->struct_size, sizeof(ssu_plan_args));
    if (!is_index(a->length_dtype) || (a->context && !is_index(a->context_dtype)) ||
        (a->block_table && !is_index(a->table_dtype)))
        return report(kBad, "length_dtype %d, context_dtype %d or table_dtype %d is not an "
                      "ssu_index_dtype", a->length_dtype, a->context_dtype, a->table_dtype);
    if (a->nseq < 0 || a->nseq > INT32_MAX || a->rows < 0 || a->rows > INT32_MAX)
        return report(kBad, "nseq %lld and rows %lld must be in [0, 2^31)", (long long)a->nseq,
                      (long long)a->rows);
    if (a->chunk_size < 0 || a->nchunks < 0 || a->nchunks > INT32_MAX ||
        (a->chunk_size == 0 && a->nchunks > 0))
        return report(kBad, "chunk_size %lld and nchunks %lld must be in [0, 2^31), and chunks need "
                      "a chunk_size", (long long)a->chunk_size, (long long)a->nchunks);
    if (a->chunk_size == 0 && (a->cu_chunk_seqlens || a->seq_idx || a->last_chunk_indices))
        return report(kBad, "chunk tables need a chunk_size");
    if (a->table_stride < 0 || a->table_width < 0 || a->block_size < 1)
        return report(kBad, "table_stride and table_width must be >= 0 and block_size >= 1");
    if (a->row_slots && !a->block_table && a->nseq > 0 && a->table_width > 0)
        return report(kBad, "row_slots needs a block_table");
    if (a->nseq > 0 && !a->lengths) return report(kBad, "lengths must not be NULL");
    const auto size = [](int32_t d) -> int64_t { return d == SSU_I64 ? 8 : 4; };
    const struct { const char* name; int64_t align; Rows rows; } in[] = {
        {"lengths", size(a->length_dtype), Rows(a->lengths, a->nseq * size(a->length_dtype))},
        {"context", size(a->context_dtype), Rows(a->context, a->nseq * size(a->context_dtype))},
        {"block_table", size(a->table_dtype),
         Rows(a->block_table, a->nseq, a->table_stride, a->table_width, size(a->table_dtype))}};
    const struct { const char* name; int64_t align; Rows rows; } written[] = {
        {"cu_seqlens", 4, Rows(a->cu_seqlens, (a->nseq + 1) * 4)},
        {"row_seq", 4, Rows(a->row_seq, a->rows * 4)},
        {"row_pos", 4, Rows(a->row_pos, a->rows * 4)},
        {"row_slots", 8, Rows(a->row_slots, a->rows * 8)},
        {"cu_chunk_seqlens", 4, Rows(a->cu_chunk_seqlens, (a->nchunks + 1) * 4)},
        {"seq_idx", 4, Rows(a->seq_idx, a->nchunks * 4)},
        {"last_chunk_indices", 4, Rows(a->last_chunk_indices, a->nseq * 4)}};
    for (const auto& x : in)
        if (!aligned(x.rows.p, x.align))
            return report(kBad, "%s must be aligned to its dtype", x.name);
    for (int i = 0; i < 7; ++i) {
        if (!aligned(written[i].rows.p, written[i].align))
            return report(kBad, "%s must be aligned to its dtype", written[i].name);
        for (const auto& x : in)
            if (overlap(written[i].rows, x.rows))
                return report(kBad, "%s overlaps %s", written[i].name, x.name);
        for (int j = 0; j < i; ++j)
            if (overlap(written[i].rows, written[j].rows))
                return report(kBad, "%s overlaps %s", written[i].name, written[j].name);
    }
    return SSU_OK;
}

}  // namespace

extern "C" int ssu_batch_plan(const ssu_plan_args* a, void* stream) {
    if (int rc = check(a)) return rc;
    PlanParams p{};
    p.lengths = a->lengths;
    p.context = a->context;
    p.table = a->block_table;
    p.cu = a->cu_seqlens;
    p.row_seq = a->row_seq;
    p.row_pos = a->row_pos;
    p.cu_chunk = a->cu_chunk_seqlens;
    p.seq_idx = a->seq_idx;
    p.last = a->last_chunk_indices;
    p.row_slots = a->row_slots;
    p.nseq = a->nseq;
    p.rows = a->rows;
    p.chunk = a->chunk_size;
    p.nchunks = a->nchunks;
    p.table_stride = a->table_stride;
    p.table_width = a->block_table ? a->table_width : 0;
    p.block_size = a->block_size;
    p.length64 = a->length_dtype == SSU_I64;
    p.context64 = a->context_dtype == SSU_I64;
    p.table64 = a->table_dtype == SSU_I64;
    const bool rows = a->row_seq || a->row_pos || a->row_slots;
    // The first workgroup writes the starts, also where there are no rows.
    int64_t row_blocks = rows ? (a->rows + kStretch - 1) / kStretch : 0;
    if (row_blocks == 0) row_blocks = 1;
    const bool chunks = a->chunk_size > 0 && (a->cu_chunk_seqlens || a->seq_idx);
    const int64_t chunk_blocks = chunks ? (a->nchunks + 1 + kStretch - 1) / kStretch : 0;
    p.row_blocks = static_cast<int32_t>(row_blocks);
    hipLaunchKernelGGL(plan_kernel, dim3(static_cast<unsigned>(row_blocks + chunk_blocks)),
                       dim3(kThreads), 0, static_cast<hipStream_t>(stream), p);
    return launched("ssu_batch_plan");
}
