"""Slots of linear attention where they are left out or their tables are empty: include/attention.h
called directly, where the Python binding refuses a call that the header allows, and the
binding's refusals."""
import ctypes

import pytest
import torch

import selective_state_update_ssu_amd as ssu
from selective_state_update_ssu_amd import _abi
from test_gpu_layer import Draw, same

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("entry,rows_of_each", [("varlen", 3), ("varlen", 700), ("update", 1), ("packed", 2)])
def test_sequences_past_the_slots_are_inert(entry, rows_of_each, delta):
    """Without a slot table sequence b uses slot b, and one that has no slot takes no part: nothing
    behind the last slot is read or written."""
    nseq, nslots, H, K, V = 5, 2, 2, 64, 40
    d, rows = Draw(3), nseq * rows_of_each
    q, k = (torch.nn.functional.normalize(d.normal(rows, H, K), dim=-1).to(DEV) for _ in range(2))
    v, decay = d.normal(rows, H, V).to(DEV), -d.uniform(0.0, 0.3, rows, H).to(DEV)
    beta = d.uniform(0.0, 1.0, rows, H).to(DEV) if delta else None
    cu = torch.arange(nseq + 1, dtype=torch.int32, device=DEV) * rows_of_each
    has = torch.ones(nseq, dtype=torch.bool, device=DEV)
    start = d.normal(nseq, H, V, K).to(DEV)  # of all sequences, though the call is told of nslots slots
    state, out = start.clone(), torch.full_like(v, float("nan"))
    a = _abi.AttentionArgs(
        struct_size=ctypes.sizeof(_abi.AttentionArgs), state_dtype=_abi.SSU_F32, state=state.data_ptr(),
        nslots=nslots, slot_stride=H * V * K, rows=rows, nheads=H, ngroups=H, key_dim=K, value_dim=V,
        q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), out=out.data_ptr(), q_stride=H * K,
        k_stride=H * K, v_stride=H * V, out_stride=H * V, io_dtype=_abi.SSU_F32,
        beta_dtype=_abi.SSU_F32, decay=decay.data_ptr(), decay_stride=H,
        beta=beta.data_ptr() if delta else None, beta_stride=H, scale=0.125, nseq=nseq,
        cu_seqlens=None if entry == "update" else cu.data_ptr(), pad_slot_id=-1)
    if entry == "varlen":
        a.has_initial = has.data_ptr()
        n = ssu.library().ssu_attention_workspace_bytes(rows, nseq, H, K, V, int(delta))
        assert (n > 0) == (rows_of_each == 700)  # uncut and cut
        workspace = torch.zeros(n + 256, dtype=torch.uint8, device=DEV)
        a.workspace = (workspace.data_ptr() + 255) // 256 * 256
        a.workspace_bytes = n
    stream = torch.cuda.current_stream().cuda_stream
    assert getattr(ssu.library(), f"ssu_attention_{entry}")(ctypes.byref(a), stream) == _abi.SSU_OK

    inert = torch.arange(nseq, dtype=torch.int32, device=DEV)
    inert[nslots:] = -1
    want_state, want = start.clone(), torch.full_like(v, float("nan"))
    kw = dict(out=want, beta=beta, scale=0.125, state_batch_indices=inert)
    if entry == "varlen":
        ssu.linear_attention_varlen(want_state, q, k, v, decay, cu, has_initial_state=has, **kw)
    elif entry == "update":
        ssu.linear_attention_update(want_state, q, k, v, decay, **kw)
    else:
        ssu.linear_attention_packed(want_state, q, k, v, decay, cu, **kw)
    kept = nslots * rows_of_each
    assert same(out[:kept], want[:kept]) and out[kept:].isnan().all()
    assert not out[:kept].isnan().any()
    assert same(state, want_state) and same(state[nslots:], start[nslots:])


@pytest.mark.parametrize("dst", [False, True])
@pytest.mark.parametrize("accepted", [False, True])
@pytest.mark.parametrize("slots", [False, True])
def test_tables_without_columns_are_refused(slots, accepted, dst):
    """Not taken for tables that are left out."""
    if not (slots or dst):
        return
    q, v, decay = torch.zeros(2, 1, 64, device=DEV), torch.zeros(2, 1, 32, device=DEV), torch.zeros(1, device=DEV)
    state = torch.zeros(2, 1, 32, 64, device=DEV)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="at least one column"):
        ssu.linear_attention_packed(
            state, q, q, v, decay, cu, state_batch_indices=table[:, :0] if slots else table,
            num_accepted_tokens=torch.ones(2, dtype=torch.int32, device=DEV) if accepted else None,
            dst_state_batch_indices=table[:, :0] if dst else None)
    assert not state.any()


def test_empty_tables_of_no_sequences():
    """Nothing to do is no error."""
    q, v = torch.zeros(0, 1, 64, device=DEV), torch.zeros(0, 1, 32, device=DEV)
    table = torch.zeros(0, 0, dtype=torch.int32, device=DEV)
    out = ssu.linear_attention_packed(
        torch.zeros(2, 1, 32, 64, device=DEV), q, q, v, torch.zeros(1, device=DEV),
        torch.zeros(1, dtype=torch.int32, device=DEV), state_batch_indices=table,
        num_accepted_tokens=torch.zeros(0, dtype=torch.int32, device=DEV), dst_state_batch_indices=table)
    assert out.shape == (0, 1, 32)
