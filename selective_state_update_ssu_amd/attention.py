"""Linear attention with a decay for each head, plain and with the delta rule: Python
binding of include/attention.h.

    linear_attention_varlen(state, q, k, v, decay, cu_seqlens, out=None, *, beta, scale,
                            has_initial_state, state_batch_indices, pad_slot_id, workspace)
    linear_attention_update(state, q, k, v, decay, out=None, *, beta, scale,
                            state_batch_indices, pad_slot_id)
    linear_attention_packed(state, q, k, v, decay, cu_seqlens, out=None, *, beta, scale,
                            num_accepted_tokens, state_batch_indices, dst_state_batch_indices,
                            pad_slot_id)

Per row t of a sequence and head h, with key head g = h // (heads // groups):

    S   = exp(decay[t, h]) * S                                S: [value_dim, key_dim]
    r   = v[t, h]                                             without beta
    r   = beta[t, h] * (v[t, h] - S @ k[t, g])                with beta (the delta rule)
    S   = S + outer(r, k[t, g]);   out[t, h] = scale * S @ q[t, g]

q and k are [rows, groups, key_dim], v and out [rows, heads, value_dim], of one type (fp32,
fp16 or bf16); rows may be strided, as columns of a wider projection are. decay holds natural
logarithms, fp32 [rows, heads] or, where it is the same for all rows, [heads]; beta is
[rows, heads], fp32 or v's type. state is [slots, heads, value_dim, key_dim] (fp32, fp16 or
bf16, its slots 16-byte aligned). key_dim is a multiple of 8 up to 256, value_dim at most 256.
q, k, v and the decays of a sequence must be finite (a decay of minus infinity forgets).

As in the other bindings, checks are host checks of shapes, dtypes, strides and devices;
kernels run on the current stream (or `stream=`); nothing is copied to the host and nothing
synchronises. There is no fallback: without the built library and binding every call raises.
"""
from __future__ import annotations

import importlib.util
import os
import threading

import torch

from . import library, library_path

__all__ = ["linear_attention_varlen", "linear_attention_update", "linear_attention_packed",
           "attention_workspace_bytes"]

_binding = None
_lock = threading.Lock()


def binding_path() -> str:
    return os.path.join(os.path.dirname(library_path()), "_serve_binding.so")


def _load():
    """The native binding (loaded on first use, after the library; raises if not built)."""
    global _binding
    with _lock:
        if _binding is None:
            library()
            if not os.path.exists(binding_path()):
                raise RuntimeError(f"{binding_path()} is not built: run "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            spec = importlib.util.spec_from_file_location("_serve_binding", binding_path())
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


def attention_workspace_bytes(rows, nseq, heads, key_dim, value_dim, delta=False):
    """Bytes a caller-provided `workspace` of linear_attention_varlen must hold: the
    library's figure plus 255, since the binding aligns the start to 256."""
    return int(library().ssu_attention_workspace_bytes(rows, nseq, heads, key_dim, value_dim,
                                                       int(bool(delta)))) + 255


def linear_attention_varlen(state, q, k, v, decay, cu_seqlens, out=None, *, beta=None, scale=1.0,
                            has_initial_state=None, state_batch_indices=None, pad_slot_id=-1,
                            workspace=None, stream=None):
    """Linear attention of packed prompts. Returns `out` [rows, heads, value_dim].

    Sequence b owns rows [cu_seqlens[b], cu_seqlens[b + 1]) and slot state_batch_indices[b]
    (None: slot b), whose state it starts from where has_initial_state (None: nowhere) is
    true, else from zeros, and which holds its last state afterwards. Rows of no sequence, and
    those of one whose slot is pad_slot_id or out of range, are not written; a
    sequence without rows leaves its slot as it is. Work goes by chunks on the matrix cores.

    Scratch: `attention_workspace_bytes(...)` bytes, taken from `workspace` (uint8) or,
    without one, allocated for the call on its stream. A caller's `workspace` serves one call
    at a time and has to outlive the graphs that recorded it."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens must be a 1-D [sequences + 1] tensor")
    return _run("attention", stream, 0, state, q, k, v, decay, cu_seqlens, out, beta, scale,
                has_initial_state, None, state_batch_indices, None, pad_slot_id, workspace)


def linear_attention_update(state, q, k, v, decay, out=None, *, beta=None, scale=1.0,
                            state_batch_indices=None, pad_slot_id=-1, stream=None):
    """The decode step: row b is one token of sequence b, whose state is slot
    state_batch_indices[b] (None: slot b), updated in place. Returns `out`."""
    return _run("attention", stream, 1, state, q, k, v, decay, None, out, beta, scale, None, None,
                state_batch_indices, None, pad_slot_id, None)


def linear_attention_packed(state, q, k, v, decay, cu_seqlens, out=None, *, beta=None, scale=1.0,
                            num_accepted_tokens=None, state_batch_indices=None,
                            dst_state_batch_indices=None, pad_slot_id=-1, stream=None):
    """A few rows per sequence with a state stored after each, as a window of drafted tokens
    needs. Returns `out`.

    Slots go as in ssu_packed_varlen: the state is read from entry num_accepted_tokens[b] - 1
    (None: 0) of row b of state_batch_indices ([sequences, steps] or flat; None: slot b), the
    state after row t of the sequence is written to entry t of dst_state_batch_indices; without
    that, the state after the last row goes to the slot that was read. Rows at and past the
    width of the tables store no state; num_accepted_tokens outside [1, width] makes
    its sequence inert."""
    return _run("attention", stream, 2, state, q, k, v, decay, cu_seqlens, out, beta, scale, None,
                num_accepted_tokens, state_batch_indices, dst_state_batch_indices, pad_slot_id,
                None)
