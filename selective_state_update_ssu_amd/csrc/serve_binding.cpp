// serve_binding.cpp -- the Python side of include/attention.h and include/batch.h: checks
// tensors, fills the argument structs and calls the library; native for the reason that
// layer_binding.cpp is. Returns new tensors only where attention.py and batch.py say so.
#include <vector>

#include "attention.h"
#include "batch.h"
#include "binding.hpp"

namespace {

using namespace binding;

Tensor scratch(PyObject* o, size_t bytes, const Tensor& like, const char* of, void** at) {
    Tensor w;
    *at = nullptr;
    if (o != Py_None) {
        w = tensor("workspace", o);
        if (w.device() != like.device() || w.scalar_type() != at::kByte || !w.is_contiguous() ||
            w.numel() < static_cast<int64_t>(bytes) + 255)
            value_error("workspace must be a contiguous uint8 tensor on " + like.device().str() +
                        " of at least " + of + "(...) = " + std::to_string(bytes + 255) + " bytes");
    } else if (bytes > 0) {
        // The call's own, freed at its end in the stream's order: the passes hand each other
        // values through it, so neither a call of another thread on this stream may write it
        // between their launches, nor may a graph that recorded them lose it.
        w = at::empty({static_cast<int64_t>(bytes) + 255}, like.options().dtype(at::kByte));
    }
    if (w.defined() && bytes > 0)
        *at = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(w.data_ptr()) + 255) / 256 * 256);
    return w;
}

// A slot table: [sequences, steps] or flat, sequence b's position t at entry b + t.
int64_t table_of(const char* name, const Tensor& t, int64_t nseq, at::Device device, int32_t* dtype,
                 int64_t* seq_stride, int64_t* step_stride) {
    if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
        value_error(std::string(name) + " must be int32 or int64, got " + name_of(t.scalar_type()));
    same_device(name, t, device);
    *dtype = t.scalar_type() == at::kLong ? SSU_I64 : SSU_I32;
    if (t.dim() == 2) {
        if (t.size(0) != nseq)
            value_error(std::string(name) + " must have one row per sequence (" +
                        std::to_string(nseq) + "), got " + list(t.sizes()));
        // (It has no storage, and the library would take it for no table.)
        if (nseq > 0 && t.size(1) < 1)
            value_error(std::string(name) + " must have at least one column, got " + list(t.sizes()));
        *seq_stride = t.stride(0);
        *step_stride = t.stride(1);
        return t.size(1);
    }
    if (t.dim() != 1 || t.size(0) < nseq)
        value_error(std::string(name) + " must be [sequences, steps] or flat [rows], got " +
                    list(t.sizes()));
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    *seq_stride = *step_stride = 1;
    return t.size(0) - nseq + 1;
}

// (entry, state, q, k, v, decay, cu_seqlens, out, beta, scale, has_initial_state, num_accepted,
//  state_batch_indices, dst_state_batch_indices, pad_slot_id, workspace) -> out;
// entry: 0 varlen, 1 update, 2 packed
PyObject* attention(PyObject* const* arg) {
    const int64_t which = integer(arg[0]);
    const bool packed = which == 2;
    const Tensor &state = tensor("state", arg[1]), &q = tensor("q", arg[2]), &k = tensor("k", arg[3]),
                 &v = tensor("v", arg[4]), &decay = tensor("decay", arg[5]),
                 &cu = optional("cu_seqlens", arg[6]), &beta = optional("beta", arg[8]),
                 &has = optional("has_initial_state", arg[10]),
                 &accepted = optional("num_accepted_tokens", arg[11]),
                 &slots = optional("state_batch_indices", arg[12]),
                 &dst = optional("dst_state_batch_indices", arg[13]);
    on_gpu("q", q);
    const at::Device device = q.device();
    const at::ScalarType io = q.scalar_type();
    if (io_code(io) < 0) unsupported("q dtype " + name_of(io) + " is not supported");
    if (io_code(state.scalar_type()) < 0)
        unsupported("state dtype " + name_of(state.scalar_type()) + " is not supported");
    if (state.dim() != 4 || q.dim() != 3 || v.dim() != 3)
        value_error("state must be [slots, heads, value_dim, key_dim], q [rows, groups, key_dim] and "
                    "v [rows, heads, value_dim], got " + list(state.sizes()) + ", " +
                    list(q.sizes()) + " and " + list(v.sizes()));
    ssu_attention_args a{};
    a.struct_size = sizeof(a);
    a.state_dtype = io_code(state.scalar_type());
    a.nslots = state.size(0);
    a.nheads = state.size(1);
    a.value_dim = state.size(2);
    a.key_dim = state.size(3);
    a.rows = q.size(0);
    a.ngroups = q.size(1);
    if (a.ngroups < 1 || a.nheads % a.ngroups)
        value_error("heads (" + std::to_string(a.nheads) + ") must be a multiple of groups (" +
                    std::to_string(a.ngroups) + ")");
    a.q_stride = rows_of("q", q, {a.rows, a.ngroups, a.key_dim}, io);
    a.k_stride = rows_of("k", k, {a.rows, a.ngroups, a.key_dim}, io);
    a.v_stride = rows_of("v", v, {a.rows, a.nheads, a.value_dim}, io);
    if (decay.dim() == 1) {
        vector("decay", decay, a.nheads, at::kFloat);
    } else {
        a.decay_stride = rows_of("decay", decay, {a.rows, a.nheads}, at::kFloat);
    }
    if (beta.defined()) {
        if (beta.scalar_type() != at::kFloat && beta.scalar_type() != io)
            value_error("beta must be fp32 or " + name_of(io) + ", got " + name_of(beta.scalar_type()));
        a.beta_stride = rows_of("beta", beta, {a.rows, a.nheads}, beta.scalar_type());
        a.beta_dtype = io_code(beta.scalar_type());
    }
    same_device("state", state, device);
    same_device("k", k, device);
    same_device("v", v, device);
    same_device("decay", decay, device);
    same_device("beta", beta, device);
    if (packed) {
        if (!cu.defined()) value_error("cu_seqlens must be a 1-D [sequences + 1] tensor");
        a.cu_dtype = ids_of("cu_seqlens", cu, device);
        if (cu.size(0) < 1) value_error("cu_seqlens must be a 1-D [sequences + 1] tensor");
        a.nseq = cu.size(0) - 1;
        a.cu_seqlens = cu.data_ptr();
        int64_t widths[2] = {0, 0};
        if (slots.defined()) {
            widths[0] = table_of("state_batch_indices", slots, a.nseq, device, &a.slot_dtype,
                                 &a.slot_seq_stride, &a.slot_step_stride);
            a.slots = slots.data_ptr();
        } else if (a.nseq > a.nslots) {
            value_error(std::to_string(a.nseq) + " sequences need as many slots without "
                        "state_batch_indices, got " + std::to_string(a.nslots));
        }
        if (dst.defined()) {
            widths[1] = table_of("dst_state_batch_indices", dst, a.nseq, device, &a.dst_dtype,
                                 &a.dst_seq_stride, &a.dst_step_stride);
            a.dst = dst.data_ptr();
        }
        if (accepted.defined()) {
            if (!slots.defined()) value_error("num_accepted_tokens needs state_batch_indices");
            if (ids_of("num_accepted_tokens", accepted, device) != a.cu_dtype)
                value_error("cu_seqlens and num_accepted_tokens must share a dtype");
            if (accepted.size(0) != a.nseq)
                value_error("num_accepted_tokens must be [" + std::to_string(a.nseq) + "], got " +
                            list(accepted.sizes()));
            a.num_accepted = accepted.data_ptr();
        }
        // The table that is stepped through bounds the steps; both do where both are.
        const int64_t read = accepted.defined() ? widths[0] : 0;
        a.steps = read && widths[1] ? (read < widths[1] ? read : widths[1]) : read + widths[1];
        if (read && widths[1] && read != widths[1])
            value_error("read and write tables have different widths " + std::to_string(read) +
                        " and " + std::to_string(widths[1]));
        if (a.steps < 1 && (accepted.defined() || dst.defined())) a.steps = 1;
    } else {
        sequences(a, cu, has, slots, a.rows, a.nslots, device);
    }
    a.slot_stride = slots_of("state", state);
    const Tensor out = [&] {
        Tensor t = arg[7] == Py_None ? at::empty({a.rows, a.nheads, a.value_dim}, v.options())
                                     : tensor("out", arg[7]);
        same_device("out", t, device);
        a.out_stride = rows_of("out", t, {a.rows, a.nheads, a.value_dim}, io);
        return t;
    }();
    a.scale = PyFloat_AsDouble(arg[9]);
    if (a.scale == -1. && PyErr_Occurred()) throw Error{nullptr, ""};
    Tensor workspace;
    if (which == 0) {
        a.workspace_bytes = ssu_attention_workspace_bytes(a.rows, a.nseq, a.nheads, a.key_dim,
                                                          a.value_dim, beta.defined());
        workspace = scratch(arg[15], a.workspace_bytes, q, "attention_workspace_bytes", &a.workspace);
    }
    a.state = state.data_ptr();
    a.q = q.data_ptr();
    a.k = k.data_ptr();
    a.v = v.data_ptr();
    a.out = out.data_ptr();
    a.decay = static_cast<const float*>(decay.data_ptr());
    a.beta = pointer(beta);
    a.io_dtype = io_code(io);
    a.pad_slot_id = integer(arg[14]);
    if (which == 0)
        call("ssu_attention_varlen", ssu_attention_varlen, a, device);
    else if (which == 1)
        call("ssu_attention_update", ssu_attention_update, a, device);
    else
        call("ssu_attention_packed", ssu_attention_packed, a, device);
    return THPVariable_Wrap(out);
}

// (target, draft_tokens, uniforms, cu_seqlens, draft_probs, temperature, workspace) ->
// (tokens, num_accepted)
PyObject* verify(PyObject* const* arg) {
    const Tensor &target = tensor("target", arg[0]), &drafts = tensor("draft_tokens", arg[1]),
                 &uniforms = tensor("uniforms", arg[2]), &cu = tensor("cu_seqlens", arg[3]),
                 &probs = optional("draft_probs", arg[4]),
                 &temperature = optional("temperature", arg[5]);
    on_gpu("target", target);
    const at::Device device = target.device();
    if (io_code(target.scalar_type()) < 0)
        unsupported("target dtype " + name_of(target.scalar_type()) + " is not supported");
    if (target.dim() != 2 || drafts.dim() != 2)
        value_error("target must be [rows, vocab] and draft_tokens [sequences, window], got " +
                    list(target.sizes()) + " and " + list(drafts.sizes()));
    ssu_verify_args a{};
    a.struct_size = sizeof(a);
    a.target_dtype = io_code(target.scalar_type());
    a.rows = target.size(0);
    a.vocab = target.size(1);
    a.nseq = drafts.size(0);
    a.window = drafts.size(1);
    if (a.vocab < 1) value_error("target must have at least one column");
    a.target_stride = rows_of("target", target, {a.rows, a.vocab}, target.scalar_type());
    if (drafts.scalar_type() != at::kInt && drafts.scalar_type() != at::kLong)
        value_error("draft_tokens must be int32 or int64, got " + name_of(drafts.scalar_type()));
    same_device("draft_tokens", drafts, device);
    a.draft_dtype = drafts.scalar_type() == at::kLong ? SSU_I64 : SSU_I32;
    a.draft_seq_stride = drafts.stride(0);
    a.draft_step_stride = drafts.stride(1);
    a.cu_dtype = ids_of("cu_seqlens", cu, device);
    if (cu.size(0) != a.nseq + 1)
        value_error("cu_seqlens must be [" + std::to_string(a.nseq + 1) + "], got " +
                    list(cu.sizes()));
    a.uniform_stride = rows_of("uniforms", uniforms, {a.nseq, a.window + 1}, at::kFloat);
    same_device("uniforms", uniforms, device);
    if (probs.defined()) {
        if (io_code(probs.scalar_type()) < 0)
            unsupported("draft_probs dtype " + name_of(probs.scalar_type()) + " is not supported");
        if (probs.sizes() != at::IntArrayRef({a.nseq, a.window, a.vocab}))
            value_error("draft_probs must be " + list({a.nseq, a.window, a.vocab}) + ", got " +
                        list(probs.sizes()));
        if (a.vocab > 1 && probs.stride(2) != 1)
            value_error("draft_probs' distributions must be contiguous, got strides " +
                        list(probs.strides()));
        same_device("draft_probs", probs, device);
        a.probs_dtype = io_code(probs.scalar_type());
        a.probs_seq_stride = probs.stride(0);
        a.probs_step_stride = probs.stride(1);
        a.draft_probs = probs.data_ptr();
    }
    vector("temperature", temperature, a.nseq, at::kFloat);
    same_device("temperature", temperature, device);
    const auto whole = at::TensorOptions().dtype(at::kInt).device(device);
    const Tensor tokens = at::empty({a.nseq, a.window + 1}, whole);
    const Tensor accepted = at::empty({a.nseq}, whole);
    a.workspace_bytes = ssu_verify_workspace_bytes(a.rows, a.nseq, a.vocab, temperature.defined());
    const Tensor workspace =
        scratch(arg[6], a.workspace_bytes, target, "verify_workspace_bytes", &a.workspace);
    a.target = target.data_ptr();
    a.drafts = drafts.data_ptr();
    a.uniforms = static_cast<const float*>(uniforms.data_ptr());
    a.temperature = static_cast<const float*>(pointer(temperature));
    a.cu_seqlens = cu.data_ptr();
    a.tokens = static_cast<int32_t*>(tokens.data_ptr());
    a.num_accepted = static_cast<int32_t*>(accepted.data_ptr());
    call("ssu_verify_drafts", ssu_verify_drafts, a, device);
    PyObject* one = THPVariable_Wrap(tokens);
    PyObject* two = THPVariable_Wrap(accepted);
    PyObject* both = one && two ? PyTuple_Pack(2, one, two) : nullptr;
    Py_XDECREF(one);
    Py_XDECREF(two);
    if (!both) throw Error{nullptr, ""};
    return both;
}

// `n` elements at byte `place` of a tensor of bytes, as a tensor.
Tensor stretch(const Tensor& whole, int64_t place, int64_t n, at::ScalarType type) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                        c10::scalarTypeToTypeMeta(type));
    c10::TensorImpl* impl = t.unsafeGetTensorImpl();
    impl->set_storage_offset(place / static_cast<int64_t>(c10::elementSize(type)));
    impl->set_sizes_contiguous({n});
    return t;
}

// (lengths, rows, chunk_size, nchunks, context_lens, block_table, block_size) -> (cu_seqlens,
// row_seq, row_pos, cu_chunk_seqlens, seq_idx, last_chunk_indices, row_slots), None for what
// is not asked for. chunk_size 0: no chunks; nchunks -1: as many as there can be
PyObject* plan(PyObject* const* arg) {
    const Tensor &lengths = tensor("lengths", arg[0]), &context = optional("context_lens", arg[4]),
                 &table = optional("block_table", arg[5]);
    on_gpu("lengths", lengths);
    const at::Device device = lengths.device();
    ssu_plan_args a{};
    a.struct_size = sizeof(a);
    a.length_dtype = ids_of("lengths", lengths, device);
    a.lengths = lengths.data_ptr();
    a.nseq = lengths.size(0);
    a.rows = integer(arg[1]);
    if (a.rows < 0 || a.rows > INT32_MAX)
        value_error("rows must be in [0, 2^31), got " + std::to_string(a.rows));
    a.chunk_size = integer(arg[2]);
    a.nchunks = integer(arg[3]);
    if (a.chunk_size < 0) value_error("chunk_size must be positive");
    if (a.nchunks < 0) a.nchunks = a.chunk_size ? a.rows / a.chunk_size + a.nseq : 0;
    if (a.nchunks > INT32_MAX) value_error("nchunks must be below 2^31");
    if (context.defined()) {
        a.context_dtype = ids_of("context_lens", context, device);
        if (context.size(0) != a.nseq)
            value_error("context_lens must be [" + std::to_string(a.nseq) + "], got " +
                        list(context.sizes()));
        a.context = context.data_ptr();
    }
    a.block_size = integer(arg[6]);
    if (a.block_size < 1) value_error("block_size must be positive");
    if (table.defined()) {
        if (table.scalar_type() != at::kInt && table.scalar_type() != at::kLong)
            value_error("block_table must be int32 or int64, got " + name_of(table.scalar_type()));
        if (table.dim() != 2 || table.size(0) != a.nseq)
            value_error("block_table must be [" + std::to_string(a.nseq) + ", blocks], got " +
                        list(table.sizes()));
        same_device("block_table", table, device);
        a.table_dtype = table.scalar_type() == at::kLong ? SSU_I64 : SSU_I32;
        a.table_stride = rows_of("block_table", table, table.sizes(), table.scalar_type());
        a.table_width = table.size(1);
        a.block_table = table.data_ptr();
    }
    // One allocation for all tables: each of its own costs as much as the launch.
    const bool chunks = a.chunk_size > 0;
    const int64_t sizes[7] = {a.nseq + 1, a.rows, a.rows, chunks ? a.nchunks + 1 : -1,
                              chunks ? a.nchunks : -1, chunks ? a.nseq : -1,
                              table.defined() ? a.rows : -1};
    const auto bytes = [&](int i) {
        return sizes[i] < 0 ? 0 : (sizes[i] * (i == 6 ? 8 : 4) + 63) / 64 * 64;
    };
    int64_t total = 0;
    for (int i = 0; i < 7; ++i) total += bytes(i);
    const Tensor whole = at::empty({total}, at::TensorOptions().dtype(at::kByte).device(device));
    void** const at[7] = {reinterpret_cast<void**>(&a.cu_seqlens), reinterpret_cast<void**>(&a.row_seq),
                          reinterpret_cast<void**>(&a.row_pos),
                          reinterpret_cast<void**>(&a.cu_chunk_seqlens),
                          reinterpret_cast<void**>(&a.seq_idx),
                          reinterpret_cast<void**>(&a.last_chunk_indices),
                          reinterpret_cast<void**>(&a.row_slots)};
    Tensor out[7];
    int64_t place = 0;
    for (int i = 0; i < 7; ++i) {
        if (sizes[i] < 0) continue;
        out[i] = stretch(whole, place, sizes[i], i == 6 ? at::kLong : at::kInt);
        *at[i] = static_cast<char*>(whole.data_ptr()) + place;
        place += bytes(i);
    }
    call("ssu_batch_plan", ssu_batch_plan, a, device);
    PyObject* tuple = PyTuple_New(7);
    if (!tuple) throw Error{nullptr, ""};
    for (int i = 0; i < 7; ++i) {
        PyObject* item = out[i].defined() ? THPVariable_Wrap(out[i]) : Py_None;
        if (item == Py_None) Py_INCREF(item);
        if (!item) {
            Py_DECREF(tuple);
            throw Error{nullptr, ""};
        }
        PyTuple_SET_ITEM(tuple, i, item);
    }
    return tuple;
}

PyMethodDef methods[] = {method<attention, 16>("attention"), method<verify, 7>("verify"),
                         method<plan, 7>("plan"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_binding() { return PyModule_Create(&module); }
