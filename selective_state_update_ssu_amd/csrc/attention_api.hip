// attention_api.hip -- the entry points of linear attention (include/attention.h): checks of
// the argument struct, the launches.
#include "attention_common.hpp"

namespace {

using namespace attention;
using layer::Rows;
using layer::aligned;
using layer::is_dtype;
using layer::is_index;
using layer::overlap;
using layer::size_of;

constexpr int64_t kAlign = 256;
int64_t round_up(int64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// How a call's sequences are cut, and its scratch. A workgroup walks one head of a piece, 64 columns
// of values, and two to four of them share a compute unit: sequences that give fewer than 512
// are cut, towards 1,024 of them, however unequal they are: a long prompt beside enough short ones is
// not. (One prompt of 32,768 rows, 80 heads of 128 x 64 in bf16, when this was chosen: 1,700 us
// uncut, 631 for 480 wanted, 580 for 1,024, 565 for 2,048.) A piece costs two more walks of its
// rows for the state, with the delta rule four and a product of matrices: short ones are
// not worth it. (4,096 rows through the delta rule, 32 heads of 128 x 128 in fp16: 508 us
// uncut, 300 with pieces of 256 rows, 270 with 512, 290 with 704.)
constexpr int64_t kWanted = 1024, kShortest = 256, kShortestDelta = 512;

struct Plan {
    int64_t piece, pieces, ends, sums, moves, total;
};

Plan plan_of(int64_t rows, int64_t nseq, int64_t nheads, int64_t K, int64_t V, bool delta) {
    Plan o{};
    const int64_t each = nheads * ((V + 63) / 64);
    o.pieces = nseq;
    if (nseq * each < kWanted / 2 && rows > 0) {
        int64_t piece = (rows * each + kWanted - 1) / kWanted;
        const int64_t shortest = delta ? kShortestDelta : kShortest;
        piece = (piece < shortest ? shortest : piece + 63) / 64 * 64;
        if (piece < rows) {
            o.piece = piece;
            o.pieces = rows / piece + nseq;
            o.sums = o.ends + round_up(o.pieces * nheads * V * K * 4);
            o.moves = o.sums;
            o.total = delta ? o.moves + round_up(o.pieces * nheads * K * K * 4)
                            : o.sums + round_up(o.pieces * nheads * 4);
        }
    }
    return o;
}

enum Entry { kVarlen, kUpdate, kPacked };

int64_t index_size(int32_t d) { return d == SSU_I64 ? 8 : 4; }

int check(const ssu_attention_args* a, Entry entry) {
    using ssu::report;
    constexpr int kBad = SSU_ERR_INVALID_ARGUMENT;
    if (!a) return report(kBad, "args must not be NULL");
    if (a->struct_size != sizeof(ssu_attention_args))
        return report(kBad, "struct_size %u != sizeof(ssu_attention_args) %zu (header mismatch)",
                      a->struct_size, sizeof(ssu_attention_args));
    if (a->reserved != 0) return report(kBad, "reserved must be 0");
    if (!is_dtype(a->state_dtype) || !is_dtype(a->io_dtype))
        return report(kBad, "state_dtype %d or io_dtype %d is not an ssu_dtype", a->state_dtype,
                      a->io_dtype);
    if (a->beta && a->beta_dtype != SSU_F32 && a->beta_dtype != a->io_dtype)
        return report(kBad, "beta must be fp32 or share the io dtype");
    if (a->rows < 0 || a->nheads < 1 || a->ngroups < 1 || a->key_dim < 1 || a->value_dim < 1 ||
        a->nslots < 1 || a->nseq < 0)
        return report(kBad,
                      "sizes must be positive (rows %lld, nheads %lld, ngroups %lld, key_dim %lld, "
                      "value_dim %lld, nslots %lld, nseq %lld)",
                      (long long)a->rows, (long long)a->nheads, (long long)a->ngroups,
                      (long long)a->key_dim, (long long)a->value_dim, (long long)a->nslots,
                      (long long)a->nseq);
    if (a->nheads % a->ngroups)
        return report(kBad, "nheads %lld must be a multiple of ngroups %lld",
                      (long long)a->nheads, (long long)a->ngroups);
    if (a->key_dim % 8 || a->key_dim > 256 || a->value_dim > 256)
        return report(SSU_ERR_UNSUPPORTED,
                      "key_dim %lld is not built (8 to 256 in steps of 8), or value_dim %lld (1 to "
                      "256)", (long long)a->key_dim, (long long)a->value_dim);
    if (a->rows > (1 << 30) || a->nseq > (1 << 30) || a->nheads > (1 << 20))
        return report(SSU_ERR_UNSUPPORTED,
                      "rows and nseq must be at most 2^30 and nheads at most 2^20");
    const int64_t slot = a->nheads * a->value_dim * a->key_dim;
    const int64_t qk = a->ngroups * a->key_dim, vo = a->nheads * a->value_dim;
    if (a->slot_stride < slot)
        return report(kBad, "slot_stride must be at least nheads * value_dim * key_dim");
    if (a->q_stride < 0 || a->k_stride < 0 || a->v_stride < 0 || a->decay_stride < 0 ||
        a->beta_stride < 0 || a->out_stride < vo)
        return report(kBad,
                      "strides must be >= 0 and out_stride at least nheads * value_dim");
    if (entry != kUpdate && !is_index(a->cu_dtype))
        return report(kBad, "cu_dtype %d is not an ssu_index_dtype", a->cu_dtype);
    if (a->slots && !is_index(a->slot_dtype))
        return report(kBad, "slot_dtype %d is not an ssu_index_dtype", a->slot_dtype);
    if (entry == kUpdate && (a->cu_seqlens || a->nseq != a->rows))
        return report(kBad, "an update has no cu_seqlens, and nseq must equal rows");
    if (entry != kVarlen && (a->has_initial || a->workspace || a->workspace_bytes))
        return report(kBad, "has_initial and workspace belong to ssu_attention_varlen");
    if (entry != kPacked && (a->num_accepted || a->dst || a->steps))
        return report(kBad, "num_accepted, dst and steps belong to ssu_attention_packed");
    if (entry == kPacked) {
        if (a->num_accepted && !a->slots)
            return report(kBad, "num_accepted needs a slot table");
        if (a->dst && !is_index(a->dst_dtype))
            return report(kBad, "dst_dtype %d is not an ssu_index_dtype", a->dst_dtype);
        if (a->slot_seq_stride < 0 || a->slot_step_stride < 0 || a->dst_seq_stride < 0 ||
            a->dst_step_stride < 0)
            return report(kBad, "table strides must be >= 0");
        if ((a->num_accepted || a->dst) && a->steps < 1)
            return report(kBad, "steps must be >= 1 with num_accepted or dst");
    }
    if (a->rows == 0 || a->nseq == 0) return SSU_OK;
    const int64_t io = size_of(a->io_dtype), st = size_of(a->state_dtype),
                  be = size_of(a->beta_dtype), cu = index_size(a->cu_dtype);
    const int64_t steps = a->steps > 0 ? a->steps : 1;
    const auto table = [&](const void* t, int64_t seq, int64_t step, int32_t dtype) {
        return Rows(t, ((a->nseq - 1) * seq + (steps - 1) * step + 1) * index_size(dtype));
    };
    const Rows slots = entry == kPacked
                           ? table(a->slots, a->slot_seq_stride, a->slot_step_stride, a->slot_dtype)
                           : Rows(a->slots, a->nseq * index_size(a->slot_dtype));
    const struct { const char* name; int64_t align; Rows rows; bool optional; } in[] = {
        {"q", io, Rows(a->q, a->rows, a->q_stride, qk, io), false},
        {"k", io, Rows(a->k, a->rows, a->k_stride, qk, io), false},
        {"v", io, Rows(a->v, a->rows, a->v_stride, vo, io), false},
        {"decay", 4, Rows(a->decay, a->rows, a->decay_stride, a->nheads, 4), false},
        {"beta", be, Rows(a->beta, a->rows, a->beta_stride, a->nheads, be), true},
        {"cu_seqlens", cu, Rows(a->cu_seqlens, (a->nseq + 1) * cu), entry == kUpdate},
        {"has_initial", 1, Rows(a->has_initial, a->nseq), true},
        {"slots", index_size(a->slot_dtype), slots, true},
        {"num_accepted", cu, Rows(a->num_accepted, a->nseq * cu), true},
        {"dst", index_size(a->dst_dtype),
         table(a->dst, a->dst_seq_stride, a->dst_step_stride, a->dst_dtype), true},
    };
    if (!a->state) return report(kBad, "state must not be NULL");
    if (!a->out) return report(kBad, "out must not be NULL");
    for (const auto& x : in) {
        if (!x.rows.p && !x.optional) return report(kBad, "%s must not be NULL", x.name);
        if (!aligned(x.rows.p, x.align))
            return report(kBad, "%s must be aligned to its dtype", x.name);
    }
    if (!aligned(a->out, io)) return report(kBad, "out must be aligned to its dtype");
    if (!aligned(a->state, 16) || a->slot_stride * st % 16)
        return report(SSU_ERR_UNSUPPORTED, "state and its slots must be 16-byte aligned");
    int64_t ws = 0;
    if (entry == kVarlen) {
        ws = static_cast<int64_t>(ssu_attention_workspace_bytes(
            a->rows, a->nseq, a->nheads, a->key_dim, a->value_dim, a->beta != nullptr));
        if (ws > 0 && (!a->workspace || !aligned(a->workspace, 256) ||
                       a->workspace_bytes < static_cast<size_t>(ws)))
            return report(kBad, "workspace must be 256-byte aligned and hold %lld bytes (got %zu)",
                          (long long)ws, a->workspace_bytes);
    }
    const struct { const char* name; Rows rows; } written[] = {
        {"out", Rows(a->out, a->rows, a->out_stride, vo, io)},
        {"state", Rows(a->state, a->nslots, a->slot_stride, slot, st)},
        {"workspace", Rows(a->workspace, ws)}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& x : in)
            if (overlap(written[i].rows, x.rows))
                return report(kBad, "%s overlaps %s", written[i].name, x.name);
        for (int j = 0; j < i; ++j)
            if (overlap(written[i].rows, written[j].rows))
                return report(kBad, "%s overlaps %s", written[i].name, written[j].name);
    }
    return SSU_OK;
}

Params params(const ssu_attention_args* a) {
    Params p{};
    p.state = a->state;
    p.q = a->q;
    p.k = a->k;
    p.v = a->v;
    p.out = a->out;
    p.decay = a->decay;
    p.beta = a->beta;
    p.cu = a->cu_seqlens;
    p.has = a->has_initial;
    p.slots = a->slots;
    p.na = a->num_accepted;
    p.dst = a->dst;
    p.nslots = a->nslots;
    p.slot_stride = a->slot_stride;
    p.rows = a->rows;
    p.nseq = a->nseq;
    p.pad_slot_id = a->pad_slot_id;
    p.q_stride = a->q_stride;
    p.k_stride = a->k_stride;
    p.v_stride = a->v_stride;
    p.out_stride = a->out_stride;
    p.decay_stride = a->decay_stride;
    p.beta_stride = a->beta_stride;
    p.slot_seq_stride = a->slot_seq_stride;
    p.slot_step_stride = a->slot_step_stride;
    p.dst_seq_stride = a->dst_seq_stride;
    p.dst_step_stride = a->dst_step_stride;
    p.steps = a->steps;
    p.scale = static_cast<float>(a->scale);
    p.nheads = static_cast<int32_t>(a->nheads);
    p.ngroups = static_cast<int32_t>(a->ngroups);
    p.per_group = p.nheads / p.ngroups;
    p.K = static_cast<int32_t>(a->key_dim);
    p.V = static_cast<int32_t>(a->value_dim);
    p.state_dtype = a->state_dtype;
    p.beta_f32 = a->beta_dtype == SSU_F32;
    p.cu64 = a->cu_dtype == SSU_I64;
    p.slot64 = a->slot_dtype == SSU_I64;
    p.dst64 = a->dst_dtype == SSU_I64;
    const int64_t io = size_of(a->io_dtype);
    // Rows of every head aligned to 16 bytes, none inside another.
    const auto wide = [&](const void* base, int64_t stride, int64_t heads, int64_t dim) {
        return aligned(base, 16) && stride * io % 16 == 0 && dim * io % 16 == 0 &&
               (a->rows <= 1 || stride >= heads * dim);
    };
    const auto near = [&](int64_t stride) { return stride < (int64_t(1) << 30) / (64 * io); };
    p.wide_qk = wide(a->q, a->q_stride, a->ngroups, a->key_dim) &&
                wide(a->k, a->k_stride, a->ngroups, a->key_dim);
    p.wide = p.wide_qk && a->rows > 1 && a->value_dim % 8 == 0 &&
             wide(a->v, a->v_stride, a->nheads, a->value_dim) &&
             wide(a->out, a->out_stride, a->nheads, a->value_dim) && near(a->q_stride) &&
             near(a->k_stride) && near(a->v_stride) && near(a->out_stride);
    return p;
}

int outcome(hipError_t e, const char* entry) {
    if (e == hipErrorInvalidConfiguration)
        return ssu::report(SSU_ERR_UNSUPPORTED, "%s: too many sequences and heads for one call",
                           entry);
    if (e != hipSuccess)
        return ssu::report(SSU_ERR_LAUNCH, "%s: launch failed: %s", entry, hipGetErrorString(e));
    return ssu::report_ok();
}

int step(const ssu_attention_args* a, bool packed, void* stream, const char* entry) {
    if (int rc = check(a, packed ? kPacked : kUpdate)) return rc;
    if (a->rows == 0 || a->nseq == 0) return ssu::report_ok();
    const Params p = params(a);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return outcome(a->io_dtype == SSU_F32   ? step_f32(p, packed, st)
                   : a->io_dtype == SSU_F16 ? step_f16(p, packed, st)
                                            : step_bf16(p, packed, st),
                   entry);
}

}  // namespace

extern "C" {

size_t ssu_attention_workspace_bytes(int64_t rows, int64_t nseq, int64_t nheads, int64_t key_dim,
                                     int64_t value_dim, int32_t delta) {
    if (rows < 0 || nseq < 0 || nheads < 1 || key_dim < 1 || value_dim < 1) return 0;
    return static_cast<size_t>(plan_of(rows, nseq, nheads, key_dim, value_dim, delta != 0).total);
}

int ssu_attention_varlen(const ssu_attention_args* a, void* stream) {
    if (int rc = check(a, kVarlen)) return rc;
    if (a->rows == 0 || a->nseq == 0) return ssu::report_ok();
    Params p = params(a);
    const Plan o = plan_of(a->rows, a->nseq, a->nheads, a->key_dim, a->value_dim, a->beta != nullptr);
    char* ws = static_cast<char*>(a->workspace);
    p.piece = o.piece;
    p.pieces = o.pieces;
    p.ends = reinterpret_cast<float*>(ws + o.ends);
    p.sums = reinterpret_cast<float*>(ws + o.sums);
    p.moves = reinterpret_cast<float*>(ws + o.moves);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return outcome(a->io_dtype == SSU_F32   ? chunk_f32(p, st)
                   : a->io_dtype == SSU_F16 ? chunk_f16(p, st)
                                            : chunk_bf16(p, st),
                   "ssu_attention_varlen");
}

int ssu_attention_update(const ssu_attention_args* a, void* stream) {
    return step(a, false, stream, "ssu_attention_update");
}

int ssu_attention_packed(const ssu_attention_args* a, void* stream) {
    return step(a, true, stream, "ssu_attention_packed");
}

}  // extern "C"
