"""The operators around the state update in a state space layer and its serving
loop: Python binding of include/layer.h.

    causal_conv1d_varlen(conv_state, x, weight, cu_seqlens, out=None, *, bias, activation,
                         has_initial_state, state_batch_indices, pad_slot_id)
    causal_conv1d_update(conv_state, x, weight, out=None, *, bias, activation,
                         state_batch_indices, pad_slot_id)
    selective_scan_varlen(state, x, dt, A, B, C, cu_seqlens, out=None, *, D, z, dt_bias,
                          dt_softplus, has_initial_state, state_batch_indices, pad_slot_id,
                          workspace)
    selective_scan_update(state, x, dt, A, B, C, out=None, *, D, z, dt_bias, dt_softplus,
                          state_batch_indices, pad_slot_id)
    cache_alloc(refcount, n), cache_free(refcount, slots), cache_retain(refcount, slots),
    cache_copy(caches, src, dst), cache_fork(caches, refcount, parents),
    cache_compact(caches, refcount)

As in the decode step's binding, checks are host checks of shapes, dtypes, strides and
devices; kernels run on the current stream (or `stream=`); nothing is copied to
the host and nothing synchronises.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from . import (_INDEX_DTYPES, _IO_DTYPES, _STATE_DTYPES, _cached_workspace, _index, _on_stream,
               _ptr, _raise, _stream, library)

__all__ = ["causal_conv1d_varlen", "causal_conv1d_update", "selective_scan_varlen",
           "selective_scan_update", "scan_workspace_bytes", "cache_alloc", "cache_free",
           "cache_retain", "cache_copy", "cache_fork", "cache_compact"]


def _on_gpu(name, device):
    if device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {device}")


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(name, t, shape, dtype):
    """Element stride between the rows of a [rows, ...] operand whose rows are dense."""
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    dense = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != dense:
            raise ValueError(f"{name}'s rows must be contiguous, got strides {t.stride()}")
        dense *= size
    # The stride of a dimension of size 1 says nothing.
    return t.stride(0) if shape[0] > 1 else dense


def _out(out, x, rows, dim):
    if out is None:
        out = torch.empty((rows, dim), dtype=x.dtype, device=x.device)
    return out, _rows("out", out, (rows, dim), x.dtype)


def _slot_dense(name, t):
    """Element stride between slots of a cache whose slots are dense inside."""
    dense = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != dense:
            raise ValueError(f"{name}'s slots must be contiguous inside, got strides {t.stride()}")
        dense *= size
    return t.stride(0) if t.shape[0] > 1 else dense


def _vector(name, t, n, dtype):
    if t is None:
        return
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be [{n}], got {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _sequences(cu_seqlens, has_initial_state, device):
    """(nseq, cu_seqlens' dtype code) of a packed call."""
    cu, code = _index("cu_seqlens", cu_seqlens, device)
    if cu is None or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu_seqlens must be a 1-D [sequences + 1] tensor")
    nseq = cu.shape[0] - 1
    if has_initial_state is not None:
        if has_initial_state.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"has_initial_state must be bool, got {has_initial_state.dtype}")
        _vector("has_initial_state", has_initial_state, nseq, has_initial_state.dtype)
    return nseq, code


def _slots(state_batch_indices, nseq, nslots, device):
    slots, code = _index("state_batch_indices", state_batch_indices, device)
    if slots is not None:
        if slots.dim() != 1 or slots.shape[0] != nseq:
            raise ValueError(f"state_batch_indices must be [{nseq}], got {list(slots.shape)}")
    elif nseq > nslots:
        raise ValueError(f"{nseq} sequences need as many slots without state_batch_indices, "
                         f"got {nslots}")
    return slots, code


def _call(entry, args, device, stream):
    lib = library()
    rc = getattr(lib, entry)(ctypes.byref(args), _stream(device, stream))
    if rc != _abi.SSU_OK:
        _raise(lib, rc, entry)


# -------------------------------------------------------------- short convolution

def _conv(entry, conv_state, x, weight, cu_seqlens, out, bias, activation, has_initial_state,
          state_batch_indices, pad_slot_id, stream):
    device = x.device
    _on_gpu("x", device)
    if x.dtype not in _IO_DTYPES:
        raise NotImplementedError(f"x dtype {x.dtype} is not supported")
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError(f"x must be [rows, dim] and weight [dim, width], got {list(x.shape)} and "
                         f"{list(weight.shape)}")
    if activation not in (None, "silu", "swish"):
        raise NotImplementedError(f"activation must be None, 'silu' or 'swish', got {activation!r}")
    rows, dim = x.shape
    width = weight.shape[1]
    if weight.shape[0] != dim or weight.dtype != x.dtype or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous {x.dtype} [{dim}, width], got "
                         f"{weight.dtype} {list(weight.shape)}")
    if not 2 <= width <= 4:
        raise NotImplementedError(f"width {width} is not built (2, 3 or 4)")
    if conv_state.dim() != 3 or tuple(conv_state.shape[1:]) != (width - 1, dim):
        raise ValueError(f"conv_state must be [slots, {width - 1}, {dim}], got "
                         f"{list(conv_state.shape)}")
    if conv_state.dtype != x.dtype:
        raise ValueError(f"conv_state must be {x.dtype}, got {conv_state.dtype}")
    _vector("bias", bias, dim, x.dtype)
    x_stride = _rows("x", x, (rows, dim), x.dtype)
    _same_device(device, conv_state=conv_state, weight=weight, bias=bias, out=out,
                 has_initial_state=has_initial_state)
    if cu_seqlens is None:
        nseq, cu_code = rows, 0
    else:
        nseq, cu_code = _sequences(cu_seqlens, has_initial_state, device)
    nslots = conv_state.shape[0]
    slots, slot_code = _slots(state_batch_indices, nseq, nslots, device)
    out, out_stride = _out(out, x, rows, dim)
    args = _abi.ConvArgs(
        ctypes.sizeof(_abi.ConvArgs), _IO_DTYPES[x.dtype], conv_state.data_ptr(), nslots,
        _slot_dense("conv_state", conv_state), x.data_ptr(), x_stride, out.data_ptr(), out_stride,
        weight.data_ptr(), _ptr(bias), rows, dim, width, activation is not None, _ptr(cu_seqlens),
        cu_code, slot_code, nseq, _ptr(has_initial_state), _ptr(slots), pad_slot_id)
    _call(entry, args, device, stream)
    return out


@_on_stream
def causal_conv1d_varlen(conv_state, x, weight, cu_seqlens, out=None, *, bias=None,
                         activation="silu", has_initial_state=None, state_batch_indices=None,
                         pad_slot_id=-1, stream=None):
    """Short causal depthwise convolution of packed prompts. Returns `out` [rows, dim].

    Sequence b owns rows [cu_seqlens[b], cu_seqlens[b + 1]) of x [rows, dim] (rows may be
    strided, as columns of a wider projection are); weight is [dim, width], width 2 to
    4, its last column meeting the row itself. conv_state [slots, width - 1, dim] holds the
    last width - 1 inputs of each slot, oldest first: the sequence starts from its
    slot's where has_initial_state (None: nowhere) is true, else from zeros, and
    leaves its own last inputs there. Rows of no sequence, and those of one whose slot is
    pad_slot_id or out of range, are not written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens must be a 1-D [sequences + 1] tensor")
    return _conv("ssu_conv1d_varlen", conv_state, x, weight, cu_seqlens, out, bias, activation,
                 has_initial_state, state_batch_indices, pad_slot_id, stream)


@_on_stream
def causal_conv1d_update(conv_state, x, weight, out=None, *, bias=None, activation="silu",
                         state_batch_indices=None, pad_slot_id=-1, stream=None):
    """The convolution's decode step: row b of x is the next input of sequence b, whose
    history is slot state_batch_indices[b] (None: slot b) and moves on by one. Returns
    `out` [batch, dim]."""
    return _conv("ssu_conv1d_update", conv_state, x, weight, None, out, bias, activation, None,
                 state_batch_indices, pad_slot_id, stream)


# ------------------------------------------------------------------ selective scan

def scan_workspace_bytes(rows, nseq, dim, dstate, ngroups):
    """Bytes a caller-provided `workspace` of selective_scan_varlen must hold: the
    library's figure plus 255, since the binding aligns the start to 256."""
    return int(library().ssu_scan_workspace_bytes(rows, nseq, dim, dstate, ngroups)) + 255


def _scan(entry, state, x, dt, A, B, C, cu_seqlens, out, D, z, dt_bias, dt_softplus,
          has_initial_state, state_batch_indices, pad_slot_id, workspace, stream):
    device = x.device
    _on_gpu("x", device)
    if x.dtype not in _IO_DTYPES:
        raise NotImplementedError(f"x dtype {x.dtype} is not supported")
    if state.dtype not in _STATE_DTYPES:
        raise NotImplementedError(f"state dtype {state.dtype} is not supported")
    if state.dim() != 3 or x.dim() != 2 or B.dim() != 3:
        raise ValueError(f"state must be [slots, dim, dstate], x [rows, dim] and B [rows, groups, "
                         f"dstate], got {list(state.shape)}, {list(x.shape)}, {list(B.shape)}")
    nslots, dim, dstate = state.shape
    rows, groups = x.shape[0], B.shape[1]
    if groups < 1 or dim % groups:
        raise ValueError(f"dim ({dim}) must be a multiple of groups ({groups})")
    if dt.dtype != torch.float32 and dt.dtype != x.dtype:
        raise ValueError(f"dt must be fp32 or {x.dtype}, got {dt.dtype}")
    if A.shape != (dim, dstate) or A.dtype != torch.float32 or not A.is_contiguous():
        raise ValueError(f"A must be a contiguous fp32 [{dim}, {dstate}], got {A.dtype} "
                         f"{list(A.shape)}")
    _vector("D", D, dim, torch.float32)
    _vector("dt_bias", dt_bias, dim, torch.float32)
    x_stride = _rows("x", x, (rows, dim), x.dtype)
    dt_stride = _rows("dt", dt, (rows, dim), dt.dtype)
    z_stride = 0 if z is None else _rows("z", z, (rows, dim), x.dtype)
    B_stride = _rows("B", B, (rows, groups, dstate), x.dtype)
    C_stride = _rows("C", C, (rows, groups, dstate), x.dtype)
    _same_device(device, state=state, dt=dt, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias, out=out,
                 has_initial_state=has_initial_state)
    ws_ptr, ws_bytes = None, 0
    if cu_seqlens is None:
        nseq, cu_code = rows, 0
    else:
        nseq, cu_code = _sequences(cu_seqlens, has_initial_state, device)
        ws_bytes = library().ssu_scan_workspace_bytes(rows, nseq, dim, dstate, groups)
        if workspace is None:
            workspace = _cached_workspace(device, ws_bytes)
        elif (workspace.device != device or workspace.dtype != torch.uint8 or
              not workspace.is_contiguous() or workspace.numel() < ws_bytes + 255):
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {device} of at "
                             f"least scan_workspace_bytes(...) = {ws_bytes + 255} bytes")
        ws_ptr = (workspace.data_ptr() + 255) // 256 * 256
    slots, slot_code = _slots(state_batch_indices, nseq, nslots, device)
    out, out_stride = _out(out, x, rows, dim)
    args = _abi.ScanArgs(
        ctypes.sizeof(_abi.ScanArgs), _STATE_DTYPES[state.dtype], state.data_ptr(), nslots,
        _slot_dense("state", state), rows, dim, dstate, groups, x.data_ptr(), _ptr(z),
        dt.data_ptr(), B.data_ptr(), C.data_ptr(), out.data_ptr(), x_stride, z_stride, dt_stride,
        B_stride, C_stride, out_stride, _IO_DTYPES[x.dtype], _IO_DTYPES[dt.dtype], A.data_ptr(),
        _ptr(D), _ptr(dt_bias), bool(dt_softplus), cu_code, _ptr(cu_seqlens), nseq,
        _ptr(has_initial_state), _ptr(slots), slot_code, 0, pad_slot_id, ws_ptr, ws_bytes)
    _call(entry, args, device, stream)
    return out


@_on_stream
def selective_scan_varlen(state, x, dt, A, B, C, cu_seqlens, out=None, *, D=None, z=None,
                          dt_bias=None, dt_softplus=False, has_initial_state=None,
                          state_batch_indices=None, pad_slot_id=-1, workspace=None, stream=None):
    """Selective scan of packed prompts with a decay per channel and state element.
    Returns `out` [rows, dim].

    x, z and dt are [rows, dim] (dt fp32 or x's dtype), B and C [rows, groups, dstate], A
    fp32 [dim, dstate], D and dt_bias fp32 [dim]; rows of x, z, dt, B and C may be
    strided. state [slots, dim, dstate] (fp32, fp16 or bf16) is read where
    has_initial_state (None: nowhere) is true and holds each sequence's last state
    afterwards. Rows of no sequence, and those of one whose slot is pad_slot_id or out of
    range, are not written.

    Scratch: `scan_workspace_bytes(...)` bytes, taken from `workspace` (uint8) or, without
    one, from the binding's buffer of this device and stream, which
    `ssd_combined_fwd_varlen` uses too and `reset_ssd_workspaces()` frees."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens must be a 1-D [sequences + 1] tensor")
    return _scan("ssu_scan_varlen", state, x, dt, A, B, C, cu_seqlens, out, D, z, dt_bias,
                 dt_softplus, has_initial_state, state_batch_indices, pad_slot_id, workspace,
                 stream)


@_on_stream
def selective_scan_update(state, x, dt, A, B, C, out=None, *, D=None, z=None, dt_bias=None,
                          dt_softplus=False, state_batch_indices=None, pad_slot_id=-1,
                          stream=None):
    """The scan's decode step: row b is one token of sequence b, whose state is slot
    state_batch_indices[b] (None: slot b), updated in place. Returns `out` [batch, dim]."""
    return _scan("ssu_scan_update", state, x, dt, A, B, C, None, out, D, z, dt_bias, dt_softplus,
                 None, state_batch_indices, pad_slot_id, None, stream)


# -------------------------------------------------------------------- cache slots

def _counts(refcount):
    _on_gpu("refcount", refcount.device)
    if refcount.dim() != 1 or refcount.dtype != torch.int32 or not refcount.is_contiguous():
        raise ValueError(f"refcount must be a contiguous int32 [slots], got {refcount.dtype} "
                         f"{list(refcount.shape)}")
    return _abi.CacheArgs(struct_size=ctypes.sizeof(_abi.CacheArgs), refcount=refcount.data_ptr(),
                          nslots=refcount.shape[0])


def _ids(name, t, device):
    if t.dim() != 1:
        raise ValueError(f"{name} must be 1-D, got {list(t.shape)}")
    return _index(name, t, device)


def _set_caches(args, caches, nslots, device):
    """Describe `caches` to the library. The host array lives as long as args."""
    blocks = (_abi.CacheBlock * len(caches))()
    for i, c in enumerate(caches):
        if c.dim() < 1 or c.shape[0] != nslots:
            raise ValueError(f"caches[{i}] must be [{nslots}, ...], got {list(c.shape)}")
        if c.device != device:
            raise ValueError(f"caches[{i}] is on {c.device}, expected {device}")
        size = c.element_size()
        numel = c.numel() // nslots if nslots else 0
        if c.is_contiguous():
            stride = numel
        else:
            stride = _slot_dense(f"caches[{i}]", c)
            if stride < numel:
                raise ValueError(f"caches[{i}]'s slots overlap, got strides {c.stride()}")
        block = blocks[i]
        block.base, block.slot_bytes, block.stride_bytes = c.data_ptr(), numel * size, stride * size
    args.caches, args.ncaches = blocks, len(caches)


@_on_stream
def cache_alloc(refcount, n, stream=None):
    """Takes the n lowest free slots (refcount 0 or below) and returns their ids, int32
    [n], ascending, -1 where no free slot is left. Each has one user afterwards."""
    args = _counts(refcount)
    if n < 0:
        raise ValueError(f"n must be >= 0, got {n}")
    ids = torch.empty((n,), dtype=torch.int32, device=refcount.device)
    args.n, args.ids = n, ids.data_ptr()
    _call("ssu_cache_alloc", args, refcount.device, stream)
    return ids


def _adjust(refcount, slots, delta, stream):
    args = _counts(refcount)
    slots, args.src_dtype = _ids("slots", slots, refcount.device)
    args.src, args.n, args.delta = slots.data_ptr(), slots.shape[0], delta
    _call("ssu_cache_adjust", args, refcount.device, stream)


@_on_stream
def cache_free(refcount, slots, stream=None):
    """Takes one user from each slot named in `slots` (as often as it is named). Slots
    without users stay free; ids out of range are skipped."""
    _adjust(refcount, slots, -1, stream)


@_on_stream
def cache_retain(refcount, slots, stream=None):
    """Adds one user to each slot in use that `slots` names (as often as it is named)."""
    _adjust(refcount, slots, 1, stream)


@_on_stream
def cache_copy(caches, src, dst, stream=None):
    """Copies slot src[i] to slot dst[i] of every cache ([slots, ...] tensors of any
    dtypes that share their slot ids). Pairs with an id out of range are skipped. A slot
    must not be a destination twice, nor a source and a destination of two pairs."""
    if not caches:
        return
    device, nslots = caches[0].device, caches[0].shape[0]
    _on_gpu("caches[0]", device)
    args = _abi.CacheArgs(struct_size=ctypes.sizeof(_abi.CacheArgs), nslots=nslots)
    _set_caches(args, caches, nslots, device)
    src, args.src_dtype = _ids("src", src, device)
    dst, args.dst_dtype = _ids("dst", dst, device)
    if src.shape != dst.shape:
        raise ValueError(f"src and dst must have as many entries, got {list(src.shape)} and "
                         f"{list(dst.shape)}")
    args.src, args.dst, args.n = src.data_ptr(), dst.data_ptr(), src.shape[0]
    _call("ssu_cache_copy", args, device, stream)


@_on_stream
def cache_fork(caches, refcount, parents, stream=None):
    """Gives every entry of `parents` (slots in use; a slot may be named several times, as
    when a prompt is answered several ways) a slot of its own with the parent's contents
    in every cache. Returns the new ids, int32, -1 where no free slot was left."""
    args = _counts(refcount)
    device = refcount.device
    _set_caches(args, caches, args.nslots, device)
    parents, args.src_dtype = _ids("parents", parents, device)
    n = parents.shape[0]
    children = torch.empty((n,), dtype=torch.int32, device=device)
    args.n, args.ids = n, children.data_ptr()
    _call("ssu_cache_alloc", args, device, stream)
    args.src, args.dst, args.dst_dtype = parents.data_ptr(), args.ids, _abi.SSU_I32
    _call("ssu_cache_copy", args, device, stream)
    return children


@_on_stream
def cache_compact(caches, refcount, stream=None):
    """Moves the slots in use to the lowest ids: with k in use, those at ids >= k move to
    the free ids below k, both in ascending order, contents and counts. Returns remap,
    int32 [slots]: a slot's new id, -1 for a free one."""
    args = _counts(refcount)
    device, nslots = refcount.device, args.nslots
    _set_caches(args, caches, nslots, device)
    remap = torch.empty((nslots,), dtype=torch.int32, device=device)
    plan = torch.empty((nslots // 2 * 2 + 1,), dtype=torch.int32, device=device)
    args.remap, args.plan = remap.data_ptr(), plan.data_ptr()
    _call("ssu_cache_compact", args, device, stream)
    return remap
