"""Draft verification where draft probabilities are no probabilities: below 0 they count as 0, and NaN
rejects its draft and leaves its token out of the draw."""
import pytest
import torch

import attention_harness as ah
import selective_state_update_ssu_amd as ssu
from test_gpu_batch import case, run

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("io", [F32, F16, BF16])
@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("vocab", [7, 1000, 20001])
def test_negative_draft_probabilities_count_as_zero(io, scores, vocab):
    c = case(vocab + 1, [3, 1, 5, 2, 4], 4, vocab, io, scores=scores, draft=True)
    c["probs"][:, :, ::3] = -c["probs"][:, :, ::3]
    c["probs"][:, 1, 1] = -INF
    at = c["probs"].argmin(-1)  # tokens below 0, drafted: the target's probability decides alone
    c["drafts"][1::2] = at[1::2].to(c["drafts"].dtype)
    zeroed = torch.where(c["probs"] < 0, torch.zeros_like(c["probs"]), c["probs"])
    tokens, counts, slack = ah.verify(c["target"], c["drafts"], c["uniforms"], c["cu"], zeroed, c["temperature"])
    assert not scores or min(slack) > 2.0 ** -35
    got, n = run(c)
    assert n.tolist() == counts and got.tolist() == tokens


def one(p, q, draft, u, drawn):
    """One sequence of one draft: the target's distributions p and (1/2, 0, 0, 1/2) behind it."""
    target = torch.tensor([p, [0.5, 0.0, 0.0, 0.5]], device=DEV)
    got, n = ssu.verify_drafts(
        target, torch.tensor([[draft]], dtype=torch.int32, device=DEV), torch.tensor([[u, drawn]], device=DEV),
        torch.tensor([0, 2], dtype=torch.int32, device=DEV), draft_probs=torch.tensor([[q]], device=DEV))
    return got.tolist()[0], int(n)


def test_draft_probabilities_by_hand():
    p = [0.0, 0.25, 0.25, 0.5]
    # A draft that the target never takes stays rejected whatever its q: the draw is from p - q.
    assert one(p, [-1.0, 0.25, 0.25, 0.25], 0, 0.5, 0.0) == ([3, -1], 1)
    # Tokens without probability gain none from a q below 0, nor do others.
    assert one(p, [-8.0, 1.0, -8.0, 0.25], 1, 0.5, 0.49) == ([2, -1], 1)
    assert one(p, [-8.0, 1.0, -8.0, 0.25], 1, 0.5, 0.5) == ([3, -1], 1)
    # q = 0 by count: the draft stands where p > 0.
    assert one(p, [0.0, -1.0, 0.0, 0.0], 1, 0.999, 0.5) == ([1, 3], 2)
    # NaN: rejected, and out of the draw.
    assert one(p, [0.0, NAN, 0.25, 0.25], 1, 0.0, 0.0) == ([3, -1], 1)
    assert one(p, [NAN, NAN, NAN, 0.75], 1, 0.0, 0.0) == ([1, -1], 1)  # nothing is left: from p
