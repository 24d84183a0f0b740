// layer_scan_api.hip -- the selective scan's entry points (include/layer.h): checks
// of the argument struct, the rule that cuts sequences into pieces, the layout of
// the scratch, the launches.
#include "layer_scan.hpp"

namespace {

using namespace layer;

constexpr int64_t kAlign = 256;
int64_t round_up(int64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

int64_t channel_blocks(int64_t dim, int64_t ngroups) {
    return (dim / ngroups + 63) / 64 * ngroups;
}

// Rows of a piece, or 0: with kEnough workgroups from the sequences alone, or none longer
// than a piece, nothing is cut. Otherwise pieces are cut so that about kWanted come to be,
// six per compute unit (1,280 to 2,560 lie within 3 %, 5,120 are 24 % slower for the joins).
// Whole against cut, 5,120 channels x 16, sequences of 1,024 rows: 144 against 53 us with 80
// workgroups (one sequence), 178 / 152 with 320, 181 / 175 with 400, 229 / 325 with 640; with
// a dstate of 64 the two meet at about 320 workgroups, with 1,024 channels at 512. The rule
// counts sequences, since their lengths are on the device: a long one beside
// empty or short ones that make up the 400 is walked whole, at 0.14 us a row.
constexpr int64_t kEnough = 400, kWanted = 1536, kShortest = 64;

int64_t piece_rows(int64_t rows, int64_t nseq, int64_t blocks) {
    if (nseq * blocks >= kEnough) return 0;
    const int64_t each = (rows * blocks + kWanted - 1) / kWanted;
    const int64_t piece = each < kShortest ? kShortest : each;
    return piece < rows ? (piece + kTile - 1) / kTile * kTile : 0;
}

struct Scratch {
    int64_t piece, pieces, ends, sums, total;
};

Scratch scratch(int64_t rows, int64_t nseq, int64_t dim, int64_t dstate, int64_t ngroups) {
    Scratch s;
    s.piece = piece_rows(rows, nseq, channel_blocks(dim, ngroups));
    s.pieces = s.piece > 0 ? rows / s.piece + nseq : nseq;
    s.ends = 0;
    s.sums = s.ends + round_up(s.piece > 0 ? s.pieces * dim * dstate * 4 : 0);
    s.total = s.sums + round_up(s.piece > 0 ? s.pieces * dim * 4 : 0);
    return s;
}

bool built(int64_t dstate) {
    return dstate == 8 || dstate == 16 || dstate == 32 || dstate == 64 || dstate == 128 ||
           dstate == 256;
}

int check(const ssu_scan_args* a, bool varlen) {
    using ssu::report;
    if (!a) return report(SSU_ERR_INVALID_ARGUMENT, "args must not be NULL");
    if (a->struct_size != sizeof(ssu_scan_args))
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "struct_size %u != sizeof(ssu_scan_args) %zu (header mismatch)",
                      a->struct_size, sizeof(ssu_scan_args));
    if (a->reserved != 0) return report(SSU_ERR_INVALID_ARGUMENT, "reserved must be 0");
    if (!is_dtype(a->state_dtype) || !is_dtype(a->io_dtype))
        return report(SSU_ERR_INVALID_ARGUMENT, "state_dtype %d or io_dtype %d is not an ssu_dtype",
                      a->state_dtype, a->io_dtype);
    if (a->dt_dtype != SSU_F32 && a->dt_dtype != a->io_dtype)
        return report(SSU_ERR_INVALID_ARGUMENT, "dt must be fp32 or share the io dtype");
    if (a->rows < 0 || a->dim < 1 || a->dim > INT32_MAX || a->ngroups < 1 || a->dstate < 1 ||
        a->nslots < 1 || a->nseq < 0)
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "sizes must be positive (rows %lld, dim %lld, dstate %lld, ngroups %lld, "
                      "nslots %lld, nseq %lld)",
                      (long long)a->rows, (long long)a->dim, (long long)a->dstate,
                      (long long)a->ngroups, (long long)a->nslots, (long long)a->nseq);
    if (a->dim % a->ngroups)
        return report(SSU_ERR_INVALID_ARGUMENT, "dim %lld must be a multiple of ngroups %lld",
                      (long long)a->dim, (long long)a->ngroups);
    if (!built(a->dstate))
        return report(SSU_ERR_UNSUPPORTED,
                      "dstate %lld is not built (8, 16, 32, 64, 128 or 256)", (long long)a->dstate);
    // The kernels count rows and a row's elements in 32 bits.
    if (a->rows > (1 << 30) || a->nseq > (1 << 30) || a->dim * a->dstate > INT32_MAX ||
        a->ngroups * a->dstate > INT32_MAX)
        return report(SSU_ERR_UNSUPPORTED,
                      "rows and nseq must be at most 2^30 and dim * dstate below 2^31");
    if (a->slot_stride < a->dim * a->dstate)
        return report(SSU_ERR_INVALID_ARGUMENT, "slot_stride must be at least dim * dstate");
    const int64_t gn = a->ngroups * a->dstate;
    if (a->x_stride < 0 || a->dt_stride < 0 || a->z_stride < 0 || a->B_stride < 0 ||
        a->C_stride < 0 || a->out_stride < a->dim)
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "strides must be >= 0 and out_stride at least dim");
    if (varlen && !is_index(a->cu_dtype))
        return report(SSU_ERR_INVALID_ARGUMENT, "cu_dtype %d is not an ssu_index_dtype",
                      a->cu_dtype);
    if (a->slots && !is_index(a->slot_dtype))
        return report(SSU_ERR_INVALID_ARGUMENT, "slot_dtype %d is not an ssu_index_dtype",
                      a->slot_dtype);
    if (!varlen && (a->cu_seqlens || a->has_initial || a->workspace || a->workspace_bytes))
        return report(SSU_ERR_INVALID_ARGUMENT,
                      "cu_seqlens, has_initial and workspace belong to ssu_scan_varlen");
    if (!varlen && a->nseq != a->rows)
        return report(SSU_ERR_INVALID_ARGUMENT, "nseq must equal rows");
    if (a->rows == 0 || a->nseq == 0) return SSU_OK;
    const int64_t io = size_of(a->io_dtype), st = size_of(a->state_dtype),
                  dt = size_of(a->dt_dtype);
    const struct { const char* name; int64_t align; Rows rows; bool optional; } in[] = {
        {"x", io, Rows(a->x, a->rows, a->x_stride, a->dim, io), false},
        {"dt", dt, Rows(a->dt, a->rows, a->dt_stride, a->dim, dt), false},
        {"B", io, Rows(a->B, a->rows, a->B_stride, gn, io), false},
        {"C", io, Rows(a->C, a->rows, a->C_stride, gn, io), false},
        {"A", 4, Rows(a->A, a->dim * a->dstate * 4), false},
        {"z", io, Rows(a->z, a->rows, a->z_stride, a->dim, io), true},
        {"D", 4, Rows(a->D, a->dim * 4), true},
        {"dt_bias", 4, Rows(a->dt_bias, a->dim * 4), true},
        {"cu_seqlens", a->cu_dtype == SSU_I64 ? 8 : 4,
         Rows(a->cu_seqlens, (a->nseq + 1) * (a->cu_dtype == SSU_I64 ? 8 : 4)), !varlen},
    };
    if (!a->state) return report(SSU_ERR_INVALID_ARGUMENT, "state must not be NULL");
    if (!a->out) return report(SSU_ERR_INVALID_ARGUMENT, "out must not be NULL");
    for (const auto& q : in) {
        if (!q.rows.p && !q.optional)
            return report(SSU_ERR_INVALID_ARGUMENT, "%s must not be NULL", q.name);
        if (!aligned(q.rows.p, q.align))
            return report(SSU_ERR_INVALID_ARGUMENT, "%s must be aligned to its dtype", q.name);
    }
    if (!aligned(a->out, io))
        return report(SSU_ERR_INVALID_ARGUMENT, "out must be aligned to its dtype");
    if (!aligned(a->state, 16) || a->slot_stride * st % 16)
        return report(SSU_ERR_UNSUPPORTED, "state and its slots must be 16-byte aligned");
    int64_t ws_bytes = 0;
    if (varlen) {
        ws_bytes = scratch(a->rows, a->nseq, a->dim, a->dstate, a->ngroups).total;
        if (ws_bytes > 0 && (!a->workspace || !aligned(a->workspace, kAlign) ||
                             a->workspace_bytes < static_cast<size_t>(ws_bytes)))
            return report(SSU_ERR_INVALID_ARGUMENT,
                          "workspace must be 256-byte aligned and hold %lld bytes (got %zu)",
                          (long long)ws_bytes, a->workspace_bytes);
    }
    const struct { const char* name; Rows rows; } written[] = {
        {"out", Rows(a->out, a->rows, a->out_stride, a->dim, io)},
        {"state", Rows(a->state, a->nslots, a->slot_stride, a->dim * a->dstate, st)},
        {"workspace", Rows(a->workspace, ws_bytes)}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& q : in)
            if (overlap(written[i].rows, q.rows))
                return report(SSU_ERR_INVALID_ARGUMENT, "%s overlaps %s", written[i].name, q.name);
        for (int j = 0; j < i; ++j)
            if (overlap(written[i].rows, written[j].rows))
                return report(SSU_ERR_INVALID_ARGUMENT, "%s overlaps %s", written[i].name,
                              written[j].name);
    }
    return SSU_OK;
}

ScanParams params(const ssu_scan_args* a) {
    ScanParams p{};
    p.state = a->state;
    p.x = a->x;
    p.z = a->z;
    p.dt = a->dt;
    p.B = a->B;
    p.C = a->C;
    p.out = a->out;
    p.A = a->A;
    p.D = a->D;
    p.dt_bias = a->dt_bias;
    p.cu = a->cu_seqlens;
    p.has = a->has_initial;
    p.slots = a->slots;
    p.nslots = a->nslots;
    p.slot_stride = a->slot_stride;
    p.rows = a->rows;
    p.nseq = a->nseq;
    p.pad_slot_id = a->pad_slot_id;
    p.x_stride = a->x_stride;
    p.z_stride = a->z_stride;
    p.dt_stride = a->dt_stride;
    p.B_stride = a->B_stride;
    p.C_stride = a->C_stride;
    p.out_stride = a->out_stride;
    p.dim = static_cast<int32_t>(a->dim);
    p.ngroups = static_cast<int32_t>(a->ngroups);
    p.group_dim = p.dim / p.ngroups;
    p.state_dtype = a->state_dtype;
    p.dt_f32 = a->dt_dtype == SSU_F32;
    p.softplus = a->dt_softplus != 0;
    p.cu64 = a->cu_dtype == SSU_I64;
    p.slot64 = a->slot_dtype == SSU_I64;
    return p;
}

int outcome(hipError_t e, const char* entry) {
    if (e != hipSuccess)
        return ssu::report(SSU_ERR_LAUNCH, "%s: launch failed: %s", entry, hipGetErrorString(e));
    return ssu::report_ok();
}

}  // namespace

extern "C" {

size_t ssu_scan_workspace_bytes(int64_t rows, int64_t nseq, int64_t dim, int64_t dstate,
                                int64_t ngroups) {
    if (rows < 0 || nseq < 0 || dim < 1 || dstate < 1 || ngroups < 1) return 0;
    return static_cast<size_t>(scratch(rows, nseq, dim, dstate, ngroups).total);
}

int ssu_scan_varlen(const ssu_scan_args* a, void* stream) {
    if (int rc = check(a, true)) return rc;
    if (a->rows == 0 || a->nseq == 0) return ssu::report_ok();
    ScanParams p = params(a);
    const Scratch s = scratch(a->rows, a->nseq, a->dim, a->dstate, a->ngroups);
    char* ws = static_cast<char*>(a->workspace);
    p.piece = s.piece;
    p.pieces = s.pieces;
    p.ends = reinterpret_cast<float*>(ws + s.ends);
    p.sums = reinterpret_cast<float*>(ws + s.sums);
    p.blocks_per_group = (p.group_dim + 63) / 64;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int n = static_cast<int>(a->dstate);
    return outcome(a->io_dtype == SSU_F32   ? scan_varlen_f32(p, n, st)
                   : a->io_dtype == SSU_F16 ? scan_varlen_f16(p, n, st)
                                            : scan_varlen_bf16(p, n, st),
                   "ssu_scan_varlen");
}

int ssu_scan_update(const ssu_scan_args* a, void* stream) {
    if (int rc = check(a, false)) return rc;
    if (a->rows == 0) return ssu::report_ok();
    ScanParams p = params(a);
    const int64_t io = size_of(a->io_dtype), st_size = size_of(a->state_dtype);
    const int each = step_channels(a->dstate, st_size);
    p.blocks_per_group = (p.group_dim + each - 1) / each;
    // A lane reads as many elements of B and C as of the state, 16 / state size.
    const int64_t bytes = 16 / st_size * io < 16 ? 16 / st_size * io : 16;
    p.wide_bc = aligned(a->B, bytes) && aligned(a->C, bytes) && a->B_stride * io % bytes == 0 &&
                a->C_stride * io % bytes == 0;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int n = static_cast<int>(a->dstate);
    return outcome(a->io_dtype == SSU_F32   ? scan_update_f32(p, n, st)
                   : a->io_dtype == SSU_F16 ? scan_update_f16(p, n, st)
                                            : scan_update_bf16(p, n, st),
                   "ssu_scan_update");
}

}  // extern "C"
