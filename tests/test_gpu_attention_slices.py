"""Prompts of bf16 rows in slices of 128 value columns (1,024 slices of 64 or more) and of 64: each
against the fp64 form, and against each other."""
import pytest
import torch

import selective_state_update_ssu_amd as ssu
from test_gpu_attention import BF16, DEV, F32, inputs, prompts
from test_gpu_layer import same

pytestmark = pytest.mark.gpu

LENGTHS = [14, 33, 31, 0, 64, 65, 16, 1, 2, 0, 0, 48, 1, 1, 15, 1, 32]


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("st", [F32, BF16])
@pytest.mark.parametrize("K,V", [(64, 128), (40, 72), (128, 128), (128, 200)])
def test_prompts_in_wide_slices(delta, st, K, V):
    c = inputs(K + V, LENGTHS, 32, 16, K, V, BF16, st, delta, lead=2, tail=3, inert=(2,), strided=False)
    assert len(LENGTHS) * 32 * -(-V // 64) >= 1024
    prompts(c)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("K,V", [(64, 128), (128, 128), (128, 200)])
def test_wide_and_narrow_slices_agree(delta, K, V):
    """A sequence alone is the same sequence among many, bit for bit."""
    c = inputs(K, LENGTHS, 32, 32, K, V, BF16, F32, delta, strided=False)
    args = [c[x].to(DEV) for x in ("q", "k", "v", "decay")]
    beta = c["beta"].to(DEV) if delta else None
    has = torch.ones(len(LENGTHS), dtype=torch.bool, device=DEV)
    slots = c["slots"].to(DEV)
    state = c["state"].to(DEV)
    out = ssu.linear_attention_varlen(state, *args, torch.tensor(c["cu"], dtype=torch.int32, device=DEV), beta=beta,
                                      scale=c["scale"], has_initial_state=has, state_batch_indices=slots)
    for b, n in enumerate(LENGTHS):
        rows = slice(c["cu"][b], c["cu"][b + 1])
        alone = c["state"].to(DEV)
        got = ssu.linear_attention_varlen(
            alone, *(x[rows] for x in args), torch.tensor([0, n], dtype=torch.int32, device=DEV),
            beta=None if beta is None else beta[rows], scale=c["scale"], has_initial_state=has[:1],
            state_batch_indices=slots[b:b + 1])
        assert same(got, out[rows])
        assert same(alone[slots[b]], state[slots[b]])
