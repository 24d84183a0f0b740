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
the host and nothing synchronises. Calls that change one `refcount` are made by one
thread at a time. The checks and the calls themselves are native
(csrc/layer_binding.cpp): a decode step of a few sequences is 4 us on the GPU, less than
filling its arguments from Python takes. There is no fallback: without the built library
and binding every call raises.
"""
from __future__ import annotations

import importlib.util
import os
import threading

import torch

from . import library, library_path

__all__ = ["causal_conv1d_varlen", "causal_conv1d_update", "selective_scan_varlen",
           "selective_scan_update", "scan_workspace_bytes", "cache_alloc", "cache_free",
           "cache_retain", "cache_copy", "cache_fork", "cache_compact"]

_binding = None
_lock = threading.Lock()


def binding_path() -> str:
    return os.path.join(os.path.dirname(library_path()), "_layer_binding.so")


def _load():
    """The native binding (loaded on first use, after the library; raises if not built)."""
    global _binding
    with _lock:
        if _binding is None:
            library()
            if not os.path.exists(binding_path()):
                raise RuntimeError(f"{binding_path()} is not built: run "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            spec = importlib.util.spec_from_file_location("_layer_binding", binding_path())
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _binding = module
    return _binding


def _run(name, stream, *args):
    f = getattr(_binding or _load(), name)
    if stream is None:
        return f(*args)
    # As the current stream, so that what the call allocates belongs to it.
    with torch.cuda.stream(stream):
        return f(*args)


# -------------------------------------------------------------- short convolution

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
    return _run("conv", stream, conv_state, x, weight, cu_seqlens, out, bias, activation,
                has_initial_state, state_batch_indices, pad_slot_id)


def causal_conv1d_update(conv_state, x, weight, out=None, *, bias=None, activation="silu",
                         state_batch_indices=None, pad_slot_id=-1, stream=None):
    """The convolution's decode step: row b of x is the next input of sequence b, whose
    history is slot state_batch_indices[b] (None: slot b) and moves on by one. Returns
    `out` [batch, dim]."""
    return _run("conv", stream, conv_state, x, weight, None, out, bias, activation, None,
                state_batch_indices, pad_slot_id)


# ------------------------------------------------------------------ selective scan

def scan_workspace_bytes(rows, nseq, dim, dstate, ngroups):
    """Bytes a caller-provided `workspace` of selective_scan_varlen must hold: the
    library's figure plus 255, since the binding aligns the start to 256."""
    return int(library().ssu_scan_workspace_bytes(rows, nseq, dim, dstate, ngroups)) + 255


def selective_scan_varlen(state, x, dt, A, B, C, cu_seqlens, out=None, *, D=None, z=None,
                          dt_bias=None, dt_softplus=False, has_initial_state=None,
                          state_batch_indices=None, pad_slot_id=-1, workspace=None, stream=None):
    """Selective scan of packed prompts with a decay per channel and state element.
    Returns `out` [rows, dim].

    x, z and dt are [rows, dim] (dt fp32 or x's dtype), B and C [rows, groups, dstate], A
    fp32 [dim, dstate], D and dt_bias fp32 [dim]; rows of x, z, dt, B and C may be
    strided. state [slots, dim, dstate] (fp32, fp16 or bf16, its slots 16-byte aligned) is read where
    has_initial_state (None: nowhere) is true and holds each sequence's last state
    afterwards. Rows of no sequence, and those of one whose slot is pad_slot_id or out of
    range, are not written.

    Scratch: `scan_workspace_bytes(...)` bytes, taken from `workspace` (uint8) or, without
    one, allocated for the call on its stream, so calls of several threads may share a
    stream and a recorded call keeps its scratch with its graph. A caller's `workspace` serves
    one call at a time and has to outlive the graphs that recorded it."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens must be a 1-D [sequences + 1] tensor")
    return _run("scan", stream, state, x, dt, A, B, C, cu_seqlens, out, D, z, dt_bias, dt_softplus,
                has_initial_state, state_batch_indices, pad_slot_id, workspace)


def selective_scan_update(state, x, dt, A, B, C, out=None, *, D=None, z=None, dt_bias=None,
                          dt_softplus=False, state_batch_indices=None, pad_slot_id=-1,
                          stream=None):
    """The scan's decode step: row b is one token of sequence b, whose state is slot
    state_batch_indices[b] (None: slot b), updated in place. Returns `out` [batch, dim]."""
    return _run("scan", stream, state, x, dt, A, B, C, None, out, D, z, dt_bias, dt_softplus, None,
                state_batch_indices, pad_slot_id, None)


# -------------------------------------------------------------------- cache slots

def cache_alloc(refcount, n, stream=None):
    """Takes the n lowest free slots (refcount 0 or below) and returns their ids, int32
    [n], ascending, -1 where no free slot is left. Each has one user afterwards."""
    return _run("cache_alloc", stream, refcount, n)


def cache_free(refcount, slots, stream=None):
    """Takes one user from each slot named in `slots` (as often as it is named). Slots
    without users stay free; ids out of range are skipped."""
    _run("cache_adjust", stream, refcount, slots, -1)


def cache_retain(refcount, slots, stream=None):
    """Adds one user to each slot in use that `slots` names (as often as it is named)."""
    _run("cache_adjust", stream, refcount, slots, 1)


def cache_copy(caches, src, dst, stream=None):
    """Copies slot src[i] to slot dst[i] of every cache ([slots, ...] tensors of any
    dtypes that share their slot ids). Pairs with an id out of range are skipped. A slot
    must not be a destination twice, nor a source and a destination of two pairs."""
    _run("cache_copy", stream, caches, src, dst)


def cache_fork(caches, refcount, parents, stream=None):
    """Gives every entry of `parents` (slots in use; a slot may be named several times, as
    when a prompt is answered several ways) a slot of its own with the parent's contents
    in every cache. Returns the new ids, int32, -1 where no free slot was left. A parent out
    of range gets a slot whose contents are left as they were."""
    return _run("cache_fork", stream, caches, refcount, parents)


def cache_compact(caches, refcount, stream=None):
    """Moves the slots in use to the lowest ids: with k in use, those at ids >= k move to
    the free ids below k, both in ascending order, contents and counts. Returns remap,
    int32 [slots]: a slot's new id, -1 for a free one."""
    return _run("cache_compact", stream, caches, refcount)
