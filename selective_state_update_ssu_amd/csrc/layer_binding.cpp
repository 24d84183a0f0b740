// layer_binding.cpp -- the Python side of include/layer.h: checks tensors, fills the
// argument structs and calls the library. It is native because the calls it serves are
// short (a decode step of a few sequences is 4 us on the GPU): reading twenty tensor
// attributes and filling a struct from Python takes longer than that.
//
// Every function raises ValueError for inconsistent arguments, NotImplementedError for
// valid ones that the library does not implement, and returns new tensors only where
// layer.py says so. Nothing here reads device data.
#include <vector>

#include "binding.hpp"
#include "layer.h"

namespace {

using namespace binding;

// (conv_state, x, weight, cu_seqlens, out, bias, activation, has_initial_state,
//  state_batch_indices, pad_slot_id) -> out
PyObject* conv(PyObject* const* arg) {
    const Tensor &state = tensor("conv_state", arg[0]), &x = tensor("x", arg[1]),
                 &weight = tensor("weight", arg[2]), &cu = optional("cu_seqlens", arg[3]),
                 &bias = optional("bias", arg[5]), &has = optional("has_initial_state", arg[7]),
                 &slots = optional("state_batch_indices", arg[8]);
    on_gpu("x", x);
    const at::Device device = x.device();
    const at::ScalarType io = x.scalar_type();
    if (io_code(io) < 0) unsupported("x dtype " + name_of(io) + " is not supported");
    if (x.dim() != 2 || weight.dim() != 2)
        value_error("x must be [rows, dim] and weight [dim, width], got " + list(x.sizes()) +
                    " and " + list(weight.sizes()));
    ssu_conv_args a{};
    a.struct_size = sizeof(a);
    a.io_dtype = io_code(io);
    if (arg[6] != Py_None) {
        const char* s = PyUnicode_Check(arg[6]) ? PyUnicode_AsUTF8(arg[6]) : "";
        if (!s) throw Error{nullptr, ""};
        if (std::string(s) != "silu" && std::string(s) != "swish")
            unsupported(std::string("activation must be None, 'silu' or 'swish', got '") + s + "'");
        a.silu = 1;
    }
    a.rows = x.size(0);
    a.dim = x.size(1);
    const int64_t width = weight.size(1);
    if (weight.size(0) != a.dim || weight.scalar_type() != io || !weight.is_contiguous())
        value_error("weight must be a contiguous " + name_of(io) + " [" + std::to_string(a.dim) +
                    ", width], got " + name_of(weight.scalar_type()) + " " + list(weight.sizes()));
    if (width < 2 || width > 4)
        unsupported("width " + std::to_string(width) + " is not built (2, 3 or 4)");
    a.width = static_cast<int32_t>(width);
    if (state.dim() != 3 || state.size(1) != width - 1 || state.size(2) != a.dim)
        value_error("conv_state must be [slots, " + std::to_string(width - 1) + ", " +
                    std::to_string(a.dim) + "], got " + list(state.sizes()));
    if (state.scalar_type() != io)
        value_error("conv_state must be " + name_of(io) + ", got " + name_of(state.scalar_type()));
    vector("bias", bias, a.dim, io);
    a.x_stride = rows_of("x", x, {a.rows, a.dim}, io);
    same_device("conv_state", state, device);
    same_device("weight", weight, device);
    same_device("bias", bias, device);
    a.nslots = state.size(0);
    sequences(a, cu, has, slots, a.rows, a.nslots, device);
    a.slot_stride = slots_of("conv_state", state);
    const Tensor out = output(arg[4], x, a.rows, a.dim, &a.out_stride);
    a.conv_state = state.data_ptr();
    a.x = x.data_ptr();
    a.out = out.data_ptr();
    a.weight = weight.data_ptr();
    a.bias = pointer(bias);
    a.pad_slot_id = integer(arg[9]);
    if (cu.defined())
        call("ssu_conv1d_varlen", ssu_conv1d_varlen, a, device);
    else
        call("ssu_conv1d_update", ssu_conv1d_update, a, device);
    return THPVariable_Wrap(out);
}

// (state, x, dt, A, B, C, cu_seqlens, out, D, z, dt_bias, dt_softplus, has_initial_state,
//  state_batch_indices, pad_slot_id, workspace) -> out
PyObject* scan(PyObject* const* arg) {
    const Tensor &state = tensor("state", arg[0]), &x = tensor("x", arg[1]),
                 &dt = tensor("dt", arg[2]), &A = tensor("A", arg[3]), &B = tensor("B", arg[4]),
                 &C = tensor("C", arg[5]), &cu = optional("cu_seqlens", arg[6]),
                 &D = optional("D", arg[8]), &z = optional("z", arg[9]),
                 &dt_bias = optional("dt_bias", arg[10]),
                 &has = optional("has_initial_state", arg[12]),
                 &slots = optional("state_batch_indices", arg[13]);
    on_gpu("x", x);
    const at::Device device = x.device();
    const at::ScalarType io = x.scalar_type();
    if (io_code(io) < 0) unsupported("x dtype " + name_of(io) + " is not supported");
    if (io_code(state.scalar_type()) < 0)
        unsupported("state dtype " + name_of(state.scalar_type()) + " is not supported");
    if (state.dim() != 3 || x.dim() != 2 || B.dim() != 3)
        value_error("state must be [slots, dim, dstate], x [rows, dim] and B [rows, groups, "
                    "dstate], got " + list(state.sizes()) + ", " + list(x.sizes()) + ", " +
                    list(B.sizes()));
    ssu_scan_args a{};
    a.struct_size = sizeof(a);
    a.state_dtype = io_code(state.scalar_type());
    a.nslots = state.size(0);
    a.dim = state.size(1);
    a.dstate = state.size(2);
    a.rows = x.size(0);
    a.ngroups = B.size(1);
    if (a.ngroups < 1 || a.dim % a.ngroups)
        value_error("dim (" + std::to_string(a.dim) + ") must be a multiple of groups (" +
                    std::to_string(a.ngroups) + ")");
    if (dt.scalar_type() != at::kFloat && dt.scalar_type() != io)
        value_error("dt must be fp32 or " + name_of(io) + ", got " + name_of(dt.scalar_type()));
    if (A.dim() != 2 || A.size(0) != a.dim || A.size(1) != a.dstate ||
        A.scalar_type() != at::kFloat || !A.is_contiguous())
        value_error("A must be a contiguous fp32 [" + std::to_string(a.dim) + ", " +
                    std::to_string(a.dstate) + "], got " + name_of(A.scalar_type()) + " " +
                    list(A.sizes()));
    vector("D", D, a.dim, at::kFloat);
    vector("dt_bias", dt_bias, a.dim, at::kFloat);
    a.x_stride = rows_of("x", x, {a.rows, a.dim}, io);
    a.dt_stride = rows_of("dt", dt, {a.rows, a.dim}, dt.scalar_type());
    a.z_stride = z.defined() ? rows_of("z", z, {a.rows, a.dim}, io) : 0;
    a.B_stride = rows_of("B", B, {a.rows, a.ngroups, a.dstate}, io);
    a.C_stride = rows_of("C", C, {a.rows, a.ngroups, a.dstate}, io);
    same_device("state", state, device);
    same_device("dt", dt, device);
    same_device("A", A, device);
    same_device("B", B, device);
    same_device("C", C, device);
    same_device("D", D, device);
    same_device("z", z, device);
    same_device("dt_bias", dt_bias, device);
    sequences(a, cu, has, slots, a.rows, a.nslots, device);
    a.slot_stride = slots_of("state", state);
    Tensor workspace;
    if (cu.defined()) {
        const size_t bytes = ssu_scan_workspace_bytes(a.rows, a.nseq, a.dim, a.dstate, a.ngroups);
        if (arg[15] != Py_None) {
            workspace = tensor("workspace", arg[15]);
            if (workspace.device() != device || workspace.scalar_type() != at::kByte ||
                !workspace.is_contiguous() ||
                workspace.numel() < static_cast<int64_t>(bytes) + 255)
                value_error("workspace must be a contiguous uint8 tensor on " + device.str() +
                            " of at least scan_workspace_bytes(...) = " +
                            std::to_string(bytes + 255) + " bytes");
        } else if (bytes > 0) {
            // The call's own, freed at its end in the stream's order: the passes hand each
            // other states through it, so neither a call of another thread on this stream may
            // write it between their launches, nor may a graph that recorded them lose it (its
            // allocations come from the graph's memory).
            workspace = at::empty({static_cast<int64_t>(bytes) + 255}, x.options().dtype(at::kByte));
        }
        if (workspace.defined()) {
            a.workspace = reinterpret_cast<void*>(
                (reinterpret_cast<uintptr_t>(workspace.data_ptr()) + 255) / 256 * 256);
            a.workspace_bytes = bytes;
        }
    }
    const Tensor out = output(arg[7], x, a.rows, a.dim, &a.out_stride);
    const int softplus = PyObject_IsTrue(arg[11]);
    if (softplus < 0) throw Error{nullptr, ""};
    a.dt_softplus = softplus;
    a.state = state.data_ptr();
    a.x = x.data_ptr();
    a.z = pointer(z);
    a.dt = dt.data_ptr();
    a.B = B.data_ptr();
    a.C = C.data_ptr();
    a.out = out.data_ptr();
    a.A = static_cast<const float*>(A.data_ptr());
    a.D = static_cast<const float*>(pointer(D));
    a.dt_bias = static_cast<const float*>(pointer(dt_bias));
    a.io_dtype = io_code(io);
    a.dt_dtype = io_code(dt.scalar_type());
    a.pad_slot_id = integer(arg[14]);
    if (cu.defined())
        call("ssu_scan_varlen", ssu_scan_varlen, a, device);
    else
        call("ssu_scan_update", ssu_scan_update, a, device);
    return THPVariable_Wrap(out);
}

// ------------------------------------------------------------------------ slots

ssu_cache_args counts(const Tensor& refcount) {
    on_gpu("refcount", refcount);
    if (refcount.dim() != 1 || refcount.scalar_type() != at::kInt || !refcount.is_contiguous())
        value_error("refcount must be a contiguous int32 [slots], got " +
                    name_of(refcount.scalar_type()) + " " + list(refcount.sizes()));
    ssu_cache_args a{};
    a.struct_size = sizeof(a);
    a.refcount = static_cast<int32_t*>(refcount.data_ptr());
    a.nslots = refcount.size(0);
    return a;
}

// A tensor is a sequence of its slots, which are no caches.
void check_list(PyObject* caches) {
    if (THPVariable_Check(caches)) value_error("caches must be a list of tensors, got a tensor");
}

std::vector<ssu_cache_block> blocks(PyObject* caches, int64_t nslots, at::Device device) {
    check_list(caches);
    PyObject* seq = PySequence_Fast(caches, "caches must be a list of tensors");
    if (!seq) throw Error{nullptr, ""};
    std::vector<ssu_cache_block> out;
    try {
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
        out.reserve(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const auto name = [i] { return "caches[" + std::to_string(i) + "]"; };
            PyObject* item = PySequence_Fast_GET_ITEM(seq, i);
            if (!THPVariable_Check(item)) value_error(name() + " must be a tensor");
            const Tensor& c = THPVariable_Unpack(item);
            if (c.dim() < 1 || c.size(0) != nslots)
                value_error(name() + " must be [" + std::to_string(nslots) + ", ...], got " +
                            list(c.sizes()));
            if (c.device() != device) same_device(name().c_str(), c, device);
            const int64_t numel = nslots ? c.numel() / nslots : 0, size = c.element_size();
            const int64_t stride = c.is_contiguous() ? numel : slots_of(name().c_str(), c);
            if (stride < numel)
                value_error(name() + "'s slots overlap, got strides " + list(c.strides()));
            out.push_back({c.data_ptr(), numel * size, stride * size});
        }
    } catch (...) {
        Py_DECREF(seq);
        throw;
    }
    Py_DECREF(seq);
    return out;
}

Tensor ids(int64_t n, at::Device device) {
    return at::empty({n}, at::TensorOptions().dtype(at::kInt).device(device));
}

// (refcount, n) -> ids
PyObject* cache_alloc(PyObject* const* arg) {
    const Tensor& refcount = tensor("refcount", arg[0]);
    ssu_cache_args a = counts(refcount);
    a.n = integer(arg[1]);
    if (a.n < 0 || a.n > INT32_MAX)
        value_error("n must be in [0, 2^31), got " + std::to_string(a.n));
    const Tensor out = ids(a.n, refcount.device());
    a.ids = static_cast<int32_t*>(out.data_ptr());
    call("ssu_cache_alloc", ssu_cache_alloc, a, refcount.device());
    return THPVariable_Wrap(out);
}

// (refcount, slots, delta)
PyObject* cache_adjust(PyObject* const* arg) {
    const Tensor &refcount = tensor("refcount", arg[0]), &slots = tensor("slots", arg[1]);
    ssu_cache_args a = counts(refcount);
    a.src_dtype = ids_of("slots", slots, refcount.device());
    a.src = slots.data_ptr();
    a.n = slots.size(0);
    a.delta = static_cast<int32_t>(integer(arg[2]));
    call("ssu_cache_adjust", ssu_cache_adjust, a, refcount.device());
    Py_RETURN_NONE;
}

// (caches, src, dst)
PyObject* cache_copy(PyObject* const* arg) {
    const Tensor &src = tensor("src", arg[1]), &dst = tensor("dst", arg[2]);
    check_list(arg[0]);
    const Py_ssize_t n = PySequence_Size(arg[0]);
    if (n < 0) throw Error{nullptr, ""};
    if (n == 0) Py_RETURN_NONE;
    PyObject* item = PySequence_GetItem(arg[0], 0);
    if (!item) throw Error{nullptr, ""};
    const bool is_tensor = THPVariable_Check(item);
    const Tensor first = is_tensor ? THPVariable_Unpack(item) : Tensor();
    Py_DECREF(item);
    if (!is_tensor || first.dim() < 1) value_error("caches[0] must be a tensor of slots");
    on_gpu("caches[0]", first);
    ssu_cache_args a{};
    a.struct_size = sizeof(a);
    a.nslots = first.size(0);
    const auto list_of = blocks(arg[0], a.nslots, first.device());
    a.caches = list_of.data();
    a.ncaches = static_cast<int64_t>(list_of.size());
    a.src_dtype = ids_of("src", src, first.device());
    a.dst_dtype = ids_of("dst", dst, first.device());
    if (src.sizes() != dst.sizes())
        value_error("src and dst must have as many entries, got " + list(src.sizes()) + " and " +
                    list(dst.sizes()));
    a.src = src.data_ptr();
    a.dst = dst.data_ptr();
    a.n = src.size(0);
    call("ssu_cache_copy", ssu_cache_copy, a, first.device());
    Py_RETURN_NONE;
}

// (caches, refcount, parents) -> children
PyObject* cache_fork(PyObject* const* arg) {
    const Tensor &refcount = tensor("refcount", arg[1]), &parents = tensor("parents", arg[2]);
    ssu_cache_args a = counts(refcount);
    const auto list_of = blocks(arg[0], a.nslots, refcount.device());
    a.caches = list_of.data();
    a.ncaches = static_cast<int64_t>(list_of.size());
    a.src_dtype = ids_of("parents", parents, refcount.device());
    a.n = parents.size(0);
    const Tensor children = ids(a.n, refcount.device());
    a.ids = static_cast<int32_t*>(children.data_ptr());
    a.src = parents.data_ptr();
    a.dst = a.ids;
    a.dst_dtype = SSU_I32;
    call("ssu_cache_alloc", ssu_cache_alloc, a, refcount.device());
    call("ssu_cache_copy", ssu_cache_copy, a, refcount.device());
    return THPVariable_Wrap(children);
}

// (caches, refcount) -> remap
PyObject* cache_compact(PyObject* const* arg) {
    const Tensor& refcount = tensor("refcount", arg[1]);
    ssu_cache_args a = counts(refcount);
    const auto list_of = blocks(arg[0], a.nslots, refcount.device());
    a.caches = list_of.data();
    a.ncaches = static_cast<int64_t>(list_of.size());
    const Tensor remap = ids(a.nslots, refcount.device());
    const Tensor plan = ids(a.nslots / 2 * 2 + 1, refcount.device());
    a.remap = static_cast<int32_t*>(remap.data_ptr());
    a.plan = static_cast<int32_t*>(plan.data_ptr());
    call("ssu_cache_compact", ssu_cache_compact, a, refcount.device());
    return THPVariable_Wrap(remap);
}

PyMethodDef methods[] = {method<conv, 10>("conv"),
                         method<scan, 16>("scan"),
                         method<cache_alloc, 2>("cache_alloc"),
                         method<cache_adjust, 3>("cache_adjust"),
                         method<cache_copy, 3>("cache_copy"),
                         method<cache_fork, 3>("cache_fork"),
                         method<cache_compact, 2>("cache_compact"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding() { return PyModule_Create(&module); }
